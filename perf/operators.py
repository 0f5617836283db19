"""Measured cases of the serving operators around the paged latent cache.

A hybrid model with Kimi Delta Attention layers keeps, for its full-attention
layers, one latent vector a token in a paged cache (absorbed latent attention),
and for its delta-rule layers one state a sequence in a slot pool.  The cases
cover what a serving step does with them:

  attn     kda_latent_attn     attention of the new tokens over the paged latents
  append   kda_latent_append   rotary positions, the new latents written into their pages
  rope     kda_rope            rotary positions on part of a head, and the gradient
  copy     kda_pages_copy      forking, reordering and clearing pages (or state slots)
  compact  kda_pages_compact   live pages moved to the front of the pool, tables renamed

With ``own`` false, run() is the operators' plain form in torch; with ``own``
true it calls the framework.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one short conversation, one token: only latency counts
        dict(name="attn_decode_1", op="attn", N=1, H=32, L=1, kv=300, page=64, dv=512, dr=64, ragged=False, varlen=False),
        # a serving batch at all stages of its conversations, one token each
        dict(name="attn_decode_64", op="attn", N=64, H=32, L=1, kv=8192, page=64, dv=512, dr=64, ragged=True, varlen=False),
        # two long documents, few heads on this GPU: the work is split along the keys
        dict(name="attn_decode_long", op="attn", N=2, H=16, L=1, kv=131071, page=128, dv=512, dr=64, ragged=False, varlen=False),
        # drafted tokens verified, four a sequence
        dict(name="attn_verify_4", op="attn", N=32, H=32, L=4, kv=8000, page=32, dv=512, dr=64, ragged=True, varlen=False),
        # chunks of prompts of different lengths behind cached prefixes
        dict(name="attn_chunk", op="attn", N=4, H=32, L=500, kv=8192, page=16, dv=512, dr=64, ragged=True, varlen=True),
        # the step's new tokens into the cache, decode and prompt chunks
        dict(name="append_decode", op="append", N=64, H=32, L=1, kv=2048, page=64, dv=512, dr=64, ragged=True, varlen=False, interleaved=True, scaled=True),
        dict(name="append_chunk", op="append", N=6, H=32, L=2047, kv=4096, page=16, dv=512, dr=64, ragged=True, varlen=True, interleaved=False, scaled=False),
        # rotary part of the queries of a prompt (the last 64 of 192 channels)
        dict(name="rope_query", op="rope", T=8192, H=32, d=192, rot=64, offset=128, far=1000000, dtype="bf16", interleaved=True, inverse=False, scaled=True),
        # its gradient, on whole heads in 32 bits
        dict(name="rope_grad_f32", op="rope", T=3001, H=8, d=128, rot=128, offset=0, far=70000, dtype="f32", interleaved=False, inverse=True, scaled=False),
        # eight sequences' delta-rule states forked into four each
        dict(name="copy_fork_states", op="copy", planes=1, pages=80, bytes=32 * 128 * 128 * 4, moves=32, sources=8, clear=4, order="fork"),
        # three latent pages of one layer: latency
        dict(name="copy_3_pages", op="copy", planes=1, pages=64, bytes=64 * 576 * 2, moves=3, sources=3, clear=0, order="shuffle"),
        # a fragmented cache of seven layers brought together
        dict(name="compact_latents", op="compact", planes=7, pages=2048, bytes=64 * 576 * 2, live=1200, listed=1600),
    ]


def _between(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "rope", "copy", "compact"])
    if op == "attn":
        H = rng.choice([1, 8, 16, 20, 32, 64, 128])
        dv = rng.choice([256, 512, 512])
        page = rng.choice([16, 32, 64, 128])
        N = _between(rng, 1, 64)
        L = _between(rng, 1, 8) if rng.random() < 0.7 else _between(rng, 9, 300)
        # rows x keys no more than the largest listed case's
        kv = _between(rng, 1, max(1, min(131072, 500000 // N, 400000000 // (N * L * H))))
        return dict(op="attn", N=N, H=H, L=L, kv=max(kv, 1), page=page, dv=dv, dr=rng.choice([0, 64, 64]),
                    ragged=rng.random() < 0.7, varlen=rng.random() < 0.4)
    if op == "append":
        N = _between(rng, 1, 64)
        L = _between(rng, 1, max(1, 6000 // N))
        return dict(op="append", N=N, H=rng.choice([1, 8, 16, 20, 32]), L=L, kv=L + _between(rng, 1, 2000),
                    page=rng.choice([16, 32, 64, 128]), dv=rng.choice([256, 512]), dr=64, ragged=rng.random() < 0.7,
                    varlen=rng.random() < 0.5, interleaved=rng.random() < 0.5, scaled=rng.random() < 0.5)
    if op == "rope":
        d = rng.choice([64, 96, 128, 192])
        rot = rng.choice([r for r in (16, 32, 64, 96, 128) if r <= d])
        return dict(op="rope", T=_between(rng, 1, 6000), H=_between(rng, 1, 32), d=d, rot=rot,
                    offset=rng.choice([0, d - rot]), far=_between(rng, 10, 1000000), dtype=rng.choice(["bf16", "f32"]),
                    interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5, scaled=rng.random() < 0.5)
    if op == "copy":
        nbytes = 16 * _between(rng, 1, 40000)
        pages = _between(rng, 4, min(2000, max(4, 200000000 // nbytes)))
        order = rng.choice(["fork", "shuffle"])
        moves = _between(rng, 1, max(1, pages // 2))
        return dict(op="copy", planes=rng.choice([1, 1, 3]), pages=pages, bytes=nbytes, moves=moves,
                    sources=_between(rng, 1, min(moves, pages - moves)) if order == "fork" else moves,
                    clear=rng.choice([0, moves // 4]) if order == "fork" else 0, order=order)
    nbytes = 16 * _between(rng, 8, 8000)
    pages = _between(rng, 8, min(4000, max(8, 200000000 // nbytes)))
    live = _between(rng, 1, pages)
    return dict(op="compact", planes=rng.choice([1, 2, 5]), pages=pages, bytes=nbytes, live=live,
                listed=live + rng.choice([0, live // 2]))


def _spread(n, top, ragged):
    """Lengths of n sequences: all `top`, or evenly spread up to it."""
    i = torch.arange(1, n + 1, dtype=torch.float64)
    return ((i / n * top).ceil() if ragged else torch.full((n,), float(top), dtype=torch.float64)).long().clamp(min=1)


def _lengths(c):
    """(new tokens, cached keys with them) of each sequence, before the seed's permutation."""
    q = _spread(c["N"], c["L"], c["varlen"])
    return q, torch.maximum(_spread(c["N"], c["kv"], c["ragged"]), q)


def work(c):
    if c["op"] == "attn":
        q, kv = _lengths(c)
        dk = c["dv"] + c["dr"]
        tokens = int(q.sum())
        pairs = int((q * kv - q * (q - 1) // 2).sum()) * c["H"]
        return {"bytes": int(kv.sum()) * dk * 2 + tokens * c["H"] * (2 * dk + 2 * c["dv"] + 4),
                "flops": 2 * pairs * (dk + c["dv"])}
    if c["op"] == "append":
        tokens = int(_lengths(c)[0].sum())
        return {"bytes": 4 * tokens * (c["dv"] + c["dr"] + c["H"] * c["dr"]),
                "flops": 3 * tokens * (c["H"] + 1) * c["dr"]}
    if c["op"] == "rope":
        n = c["T"] * c["H"] * c["d"]
        return {"bytes": 2 * n * (2 if c["dtype"] == "bf16" else 4) + 4 * c["T"], "flops": 3 * c["T"] * c["H"] * c["rot"]}
    if c["op"] == "copy":
        return {"bytes": c["planes"] * c["bytes"] * (c["sources"] + c["moves"]), "flops": 0}
    # about as many pages move as there are holes in front: live * (1 - live / pages)
    return {"bytes": 2 * c["planes"] * c["bytes"] * max(1, int(c["live"] * (1 - c["live"] / c["pages"]))) + 8 * c["listed"],
            "flops": 0}


# ------------------------------------------------------------------ inputs
def _freqs(rot, scaled):
    """Radians a position of each rotated pair; `scaled`: stretched for long
    contexts, the slow pairs by 8 and the fast ones not at all."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaled:
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        f = f * keep + f / 8 * (1 - keep)
    return f.float().to(DEV)


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=DEV).to(dtype)

    s = dict(c)
    if c["op"] in ("attn", "append"):
        ql, kv = _lengths(c)
        order = torch.randperm(c["N"], generator=cpu)
        ql, kv = ql[order], kv[order]
        dk, T = c["dv"] + c["dr"], int(ql.sum())
        per = (kv + c["page"] - 1) // c["page"]
        total, width = int(per.sum()), int(per.max())
        ids = torch.randperm(total + 3, generator=cpu)[:total].int()
        table = torch.full((c["N"], width), -1, dtype=torch.int32)
        table[torch.arange(width)[None, :] < per[:, None]] = ids
        s["table"], s["kv_lens"] = table.to(DEV), kv.int().to(DEV)
        s["cu"] = torch.cat([torch.zeros(1, dtype=torch.long), ql.cumsum(0)]).int().to(DEV) if c["varlen"] else None
        s["T"], s["max_q"], s["max_kv"] = T, int(ql.max()), int(kv.max())
        s["cache"] = randn(total + 3, c["page"], dk)
        if c["op"] == "attn":
            s["q"] = randn(T, c["H"], dk)
            # logits of about 1.7 in standard deviation, as trained heads have
            s["scale"] = 0.0722 * math.sqrt(576 / dk)
        else:
            s["kv"] = randn(T, dk)
            # the rotary part is a slice of the projection's output
            s["q_pe"] = randn(T, c["H"], 128 + c["dr"])[..., 128:]
            s["q"] = randn(T, c["H"], dk)
            s["freqs"] = _freqs(c["dr"], c["scaled"])
            s["scale"] = 1.0 + 0.1 * math.log(8) if c["scaled"] else 1.0
    elif c["op"] == "rope":
        s["x"] = randn(c["T"], c["H"], c["d"], dtype=DTYPES[c["dtype"]])
        s["positions"] = torch.randint(0, c["far"], (c["T"],), generator=g, device=DEV, dtype=torch.int32)
        s["freqs"] = _freqs(c["rot"], c["scaled"])
        s["scale"] = 1.0 + 0.1 * math.log(8) if c["scaled"] else 1.0
    else:
        s["pool"] = randn(c["planes"], c["pages"], c["bytes"] // 4, dtype=torch.float32)
        perm = torch.randperm(c["pages"], generator=cpu)
        if c["op"] == "copy":
            if c["order"] == "fork":        # each source into several fresh pages, some pages cleared
                dst = perm[:c["moves"]]
                src = perm[c["moves"]:c["moves"] + c["sources"]].repeat(-(-c["moves"] // c["sources"]))[:c["moves"]].clone()
                src[:c["clear"]] = -1
            else:                           # pages change places with one another
                dst = perm[:c["moves"]]
                src = dst[torch.randperm(c["moves"], generator=cpu)]
            s["src"], s["dst"] = src.int().to(DEV), dst.int().to(DEV)
        else:                               # some live pages are listed twice (shared prefixes), some entries are padding
            live = perm[:c["live"]]
            more = c["listed"] - c["live"]
            pages = torch.cat([live, live[:more // 2], torch.full((more - more // 2,), -1, dtype=torch.long)])
            s["listed_pages"] = pages[torch.randperm(len(pages), generator=cpu)].int().to(DEV)
    torch.cuda.synchronize()
    return s


# ------------------------------------------------------------------ plain forms
def _token_places(s):
    """(sequence, place among its new tokens, position) of each new token."""
    t = torch.arange(s["T"], device=DEV)
    if s["cu"] is None:
        each = s["T"] // s["N"]
        seq, at = t // each, t % each
        count = torch.full_like(seq, each)
    else:
        cu = s["cu"].long()
        seq = torch.bucketize(t, cu[1:], right=True)
        at, count = t - cu[seq], cu[seq + 1] - cu[seq]
    return seq, at, s["kv_lens"].long()[seq] - count + at


def _plain_attn(s):
    dv, H, page = s["dv"], s["H"], s["page"]
    dk = s["cache"].shape[-1]
    seq, at, pos = _token_places(s)
    keys = torch.arange(s["max_kv"], device=DEV)
    rows = s["table"].long()[:, keys // page] * page + keys % page
    valid = keys[None, :] < s["kv_lens"][:, None]
    k = s["cache"].view(-1, dk)[torch.where(valid, rows, 0)].float()
    k = torch.where(valid[..., None], k, 0.0)
    q = torch.zeros(s["N"], s["max_q"], H, dk, device=DEV)
    q[seq, at] = s["q"].float()
    reach = torch.full((s["N"], s["max_q"]), -1, dtype=torch.long, device=DEV)
    reach[seq, at] = pos
    x = torch.bmm(q.view(s["N"], -1, dk), k.transpose(1, 2)).view(s["N"], s["max_q"], H, -1) * s["scale"]
    x = x.masked_fill_((keys[None, None, :] > reach[..., None])[:, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(s["N"], -1, p.shape[-1]), k[..., :dv]).view(s["N"], s["max_q"], H, dv)
    o = o / torch.where(total > 0, total, 1.0)
    lse = (m + total.log())[..., 0]
    return {"out": o[seq, at].to(torch.bfloat16), "lse": lse[seq, at]}


def _rotate(x, angles, interleaved, sign, scale):
    """Pairs of the last dimension turned by `angles` (64 bits, per token)."""
    cos, sin = (angles.cos() * scale).float(), (angles.sin() * (sign * scale)).float()
    cos, sin = cos[:, None, :], sin[:, None, :]
    x = x.float()
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _plain_append(s):
    dv, page = s["dv"], s["page"]
    seq, _, pos = _token_places(s)
    angles = pos.double()[:, None] * s["freqs"].double()[None, :]
    row = s["table"].long()[seq, pos // page] * page + pos % page
    k_pe = _rotate(s["kv"][:, None, dv:], angles, s["interleaved"], 1.0, s["scale"])[:, 0]
    flat = s["cache"].view(-1, s["cache"].shape[-1])
    flat[row] = torch.cat([s["kv"][:, :dv], k_pe.to(torch.bfloat16)], -1)
    s["q"][..., dv:] = _rotate(s["q_pe"], angles, s["interleaved"], 1.0, s["scale"]).to(torch.bfloat16)
    return {"cache": s["cache"], "q": s["q"]}


def _plain_rope(s):
    a, b = s["offset"], s["offset"] + s["rot"]
    angles = s["positions"].double()[:, None] * s["freqs"].double()[None, :]
    y = s["x"].clone()
    y[..., a:b] = _rotate(s["x"][..., a:b], angles, s["interleaved"], -1.0 if s["inverse"] else 1.0, s["scale"]).to(y.dtype)
    return {"y": y}


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    got = s["pool"][:, src.clamp(min=0)]
    s["pool"][:, dst] = torch.where((src >= 0)[None, :, None], got, 0.0)
    return {"pool": s["pool"]}


def _plain_compact(s):
    pages = s["listed_pages"].long()
    n = s["pages"]
    live = torch.zeros(n + 1, dtype=torch.bool, device=DEV)
    live[torch.where(pages >= 0, pages, n)] = True
    live = live[:n]
    front = torch.arange(n, device=DEV) < live.sum()
    holes, movers = torch.nonzero(front & ~live)[:, 0], torch.nonzero(live & ~front)[:, 0]
    name = torch.arange(n, device=DEV)
    name[movers] = holes
    s["pool"][:, holes] = s["pool"][:, movers]
    return {"pool": s["pool"], "pages": torch.where(pages >= 0, name[pages.clamp(min=0)], -1).int()}


def run(s):
    op = s["op"]
    if not own:
        return {"attn": _plain_attn, "append": _plain_append, "rope": _plain_rope, "copy": _plain_copy,
                "compact": _plain_compact}[op](s)
    import gated_delta_rule_88_b200 as kda
    if op == "attn":
        out, lse = kda.kda_latent_attn(s["q"], s["cache"], s["table"], s["kv_lens"], dv=s["dv"], cu_seqlens=s["cu"],
                                       scale=s["scale"])
        return {"out": out, "lse": lse}
    if op == "append":
        kda.kda_latent_append(s["kv"], s["cache"], s["table"], s["kv_lens"], q_pe=s["q_pe"], q=s["q"], freqs=s["freqs"],
                              cu_seqlens=s["cu"], interleaved=s["interleaved"], scale=s["scale"])
        return {"cache": s["cache"], "q": s["q"]}
    if op == "rope":
        return {"y": kda.kda_rope(s["x"], s["positions"], s["freqs"], offset=s["offset"], interleaved=s["interleaved"],
                                  inverse=s["inverse"], scale=s["scale"])}
    if op == "copy":
        kda.kda_pages_copy(s["pool"], s["src"], s["dst"], planes=True)
        return {"pool": s["pool"]}
    return {"pool": s["pool"], "pages": kda.kda_pages_compact(s["pool"], s["listed_pages"], planes=True)}


# ------------------------------------------------------------------ 64 bits
def _turn64(x, pos, freqs, c, sign):
    """Complex rotation of the last dimension's pairs, in 64 bits."""
    x = x.double()
    half = x.shape[-1] // 2
    z = torch.view_as_complex(x.reshape(*x.shape[:-1], half, 2).contiguous()) if c["interleaved"] else \
        torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous())
    phase = sign * pos.double()[:, None] * freqs.double()[None, :]
    z = z * torch.polar(torch.ones_like(phase), phase)[:, None, :]
    return torch.view_as_real(z).flatten(-2) if c["interleaved"] else torch.cat([z.real, z.imag], -1)


def exact(c, seed):
    if c["op"] in ("copy", "compact"):
        return None                       # values are moved, not computed
    s = prepare(c, seed)
    if c["op"] == "rope":
        y = s["x"].double()
        a, b = c["offset"], c["offset"] + c["rot"]
        y[..., a:b] = s["scale"] * _turn64(s["x"][..., a:b], s["positions"], s["freqs"], c, -1 if c["inverse"] else 1)
        return {"y": y}
    N, page, dv, dk = c["N"], c["page"], c["dv"], c["dv"] + c["dr"]
    kv = s["kv_lens"].tolist()
    cu = s["cu"].tolist() if s["cu"] is not None else [i * (s["T"] // N) for i in range(N + 1)]
    if c["op"] == "append":
        cache, q = s["cache"].double(), s["q"].double()
        for n in range(N):
            new = slice(cu[n], cu[n + 1])
            pos = torch.arange(kv[n] - (cu[n + 1] - cu[n]), kv[n], device=DEV)
            at = s["table"][n].long()[pos // page], pos % page
            cache[at[0], at[1], :dv] = s["kv"][new, :dv].double()
            cache[at[0], at[1], dv:] = s["scale"] * _turn64(s["kv"][new, None, dv:], pos, s["freqs"], c, 1)[:, 0]
            q[new, :, dv:] = s["scale"] * _turn64(s["q_pe"][new], pos, s["freqs"], c, 1)
        return {"cache": cache, "q": q}
    out = torch.empty(s["T"], c["H"], dv, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["T"], c["H"], dtype=torch.float64, device=DEV)
    for n in range(N):
        k = s["cache"][s["table"][n].long().clamp(min=0)].reshape(-1, dk)[:kv[n]].double()
        count = cu[n + 1] - cu[n]
        step = max(1, 200_000_000 // (c["H"] * max(1, kv[n])))
        for t0 in range(0, count, step):
            t1 = min(count, t0 + step)
            x = torch.einsum("thd,kd->thk", s["q"][cu[n] + t0:cu[n] + t1].double(), k) * s["scale"]
            last = kv[n] - count + torch.arange(t0, t1, device=DEV)
            x = x.masked_fill(torch.arange(kv[n], device=DEV)[None, None, :] > last[:, None, None], -math.inf)
            out[cu[n] + t0:cu[n] + t1] = torch.einsum("thk,kd->thd", torch.softmax(x, -1), k[:, :dv])
            lse[cu[n] + t0:cu[n] + t1] = torch.logsumexp(x, -1)
    return {"out": out, "lse": lse}
