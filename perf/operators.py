"""The operators around attention that are measured: per-head norms and position rotation
of queries and keys (forward, backward, and into a paged cache), block tables and slot maps
of a paged cache, and the attention of new tokens over it.

``run`` computes a case in plain torch operations, or through the framework's entry
points where ``own`` is true. A layer's sizes are those of the framework's video workloads
(40 heads, or 24 query heads over 8 key heads, of 128; frames of 30 x 52 tokens, 21 of them
in a clip) and of its small tests (heads of 64).
"""

import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FRAME = 30 * 52          # tokens of one latent frame
CLIP = 21 * FRAME        # tokens of a clip (32760)

# What the largest listed case costs; a drawn case stays below.
MAX_FLOPS = 1.0e12
MAX_BYTES = 2.9e9


# ------------------------------------------------------------------ cases
def listed():
    return [
        # every query and key of a clip, sliced out of a fused projection, before the
        # sparse attention of one layer
        dict(name="norm_clip", op="norm", dtype="bf16", B=1, Hq=40, Hkv=40, S=CLIP, D=128,
             interleaved=True, layout="fused"),
        # the smallest workload's tensors in fp32: latency counts
        dict(name="norm_small_f32", op="norm", dtype="f32", B=1, Hq=2, Hkv=2, S=1024, D=64,
             interleaved=False, layout="heads"),
        # training: gradients of a clip's layer with shared key heads
        dict(name="norm_back_clip", op="norm_back", dtype="bf16", B=1, Hq=24, Hkv=8, S=32768, D=128,
             interleaved=True, layout="tokens"),
        # training on short odd sequences
        dict(name="norm_back_short", op="norm_back", dtype="f16", B=3, Hq=8, Hkv=2, S=333, D=64,
             interleaved=False, layout="tokens"),
        # a generated frame enters the cache
        dict(name="append_frame", op="append", dtype="bf16", Hq=24, Hkv=8, D=128, page=64,
             interleaved=True, R=1, context=20 * FRAME, chunk=FRAME, lens=1),
        # one token of each of 64 requests enters the cache
        dict(name="append_tokens", op="append", dtype="bf16", Hq=24, Hkv=8, D=128, page=16,
             interleaved=False, R=64, context=8192, chunk=1, lens=2),
        # a single request takes its next token
        dict(name="tables_token", op="tables", page=16, R=1, context=4000, chunk=1, lens=3),
        # a batch of chunks between one token and a frame
        dict(name="tables_batch", op="tables", page=64, R=256, context=CLIP, chunk=FRAME, lens=4),
        # one token over a long cache
        dict(name="attend_token", op="attend", dtype="bf16", Hq=24, Hkv=8, D=128, page=64, R=1,
             context=CLIP, chunk=1, causal=True, keep=1.0, lens=5),
        # one token of each of 64 requests, ragged contexts
        dict(name="attend_tokens", op="attend", dtype="bf16", Hq=24, Hkv=8, D=128, page=16, R=64,
             context=CLIP, chunk=1, causal=True, keep=1.0, lens=6),
        # the clip's last frame over the twenty before it, one layer
        dict(name="attend_frame", op="attend", dtype="bf16", Hq=40, Hkv=40, D=128, page=128, R=1,
             context=20 * FRAME, chunk=FRAME, causal=False, keep=1.0, lens=7),
        # chunks of several lengths with a page mask that keeps two pages of five
        dict(name="attend_masked", op="attend", dtype="f16", Hq=16, Hkv=4, D=64, page=32, R=7,
             context=8192, chunk=600, causal=True, keep=0.4, lens=8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["norm", "norm_back", "append", "tables", "attend", "attend"])
        Hq, Hkv = rng.choice([(40, 40), (24, 8), (2, 2), (8, 2), (16, 4), (6, 1), (5, 5)])
        D = rng.choice([64, 128])
        page = rng.choice([16, 32, 64, 128])
        lens = rng.randrange(1 << 30)
        if op in ("norm", "norm_back"):
            case = dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), B=rng.choice([1, 1, 2, 3]),
                        Hq=Hq, Hkv=Hkv, S=_log_int(rng, 1, CLIP), D=D,
                        interleaved=rng.random() < 0.5,
                        layout=rng.choice(["heads", "tokens", "fused"]))
        elif op == "append":
            case = dict(op=op, dtype=rng.choice(["bf16", "f16"]), Hq=Hq, Hkv=Hkv, D=D, page=page,
                        interleaved=rng.random() < 0.5, R=_log_int(rng, 1, 64),
                        context=_log_int(rng, 1, 8192), chunk=_log_int(rng, 1, FRAME), lens=lens)
        elif op == "tables":
            case = dict(op=op, page=page, R=_log_int(rng, 1, 512), context=_log_int(rng, 1, CLIP),
                        chunk=_log_int(rng, 1, FRAME), lens=lens)
        else:
            case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16"]), Hq=Hq, Hkv=Hkv, D=D,
                        page=page, R=_log_int(rng, 1, 64), context=_log_int(rng, 1, CLIP),
                        chunk=rng.choice([1, 1, _log_int(rng, 1, FRAME)]),
                        causal=rng.random() < 0.5, keep=rng.choice([1.0, 1.0, 0.4]), lens=lens)
        w = work(case)
        if w["flops"] <= MAX_FLOPS and w["bytes"] <= MAX_BYTES:
            return case


def _lengths(case):
    """Context and new-token counts of the requests: one request has the case's own
    numbers; several have contexts from 0 to the case's and chunks from 1 to it."""
    R, context, chunk = case["R"], case["context"], case["chunk"]
    if R == 1:
        return [context], [chunk]
    g = random.Random(case["lens"])
    ctx = [int(context * g.random() ** 2) for _ in range(R)]
    new = [g.randint(1, chunk) for _ in range(R)]
    return ctx, new


def _kept_pages(case):
    """bool (R, Hkv, pages of the longest request): the pages a request's KV head keeps."""
    ctx, new = _lengths(case)
    width = max(-(-(c + n) // case["page"]) for c, n in zip(ctx, new))
    if case["keep"] >= 1.0:
        return None
    g = np.random.default_rng(case["lens"])
    return g.random((case["R"], case["Hkv"], width)) < case["keep"]


def work(case):
    op = case["op"]
    if op in ("norm", "norm_back"):
        es = 4 if case["dtype"] == "f32" else 2
        rows = case["B"] * case["S"] * (case["Hq"] + case["Hkv"])
        n = rows * case["D"]
        table = 4 * case["S"] * case["D"]
        if op == "norm":
            return {"bytes": 2 * es * n + table, "flops": 9 * n}
        return {"bytes": 3 * es * n + table, "flops": 20 * n}
    ctx, new = _lengths(case)
    T = sum(new)
    if op == "append":
        D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
        n = T * (Hq + Hkv) * D
        return {"bytes": 2 * 2 * (n + T * Hkv * D) + T * (4 * D + 8), "flops": 9 * n}
    if op == "tables":
        P = case["page"]
        taken = sum(-(-(c + n) // P) - -(-c // P) for c, n in zip(ctx, new))
        return {"bytes": 8 * T + 12 * case["R"] + 8 * taken, "flops": 4 * T}
    D, Hq, Hkv, P = case["D"], case["Hq"], case["Hkv"], case["page"]
    keep = _kept_pages(case)
    keys = pairs = pages = 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        L = c + n
        np_ = -(-L // P)
        pages += np_
        size = np.full(np_, P)
        size[-1] = L - (np_ - 1) * P
        kept = np.ones((Hkv, np_), bool) if keep is None else keep[r, :, :np_]
        keys += int((kept * size).sum())
        full = n * L if not case["causal"] else n * c + n * (n + 1) // 2
        if keep is None:
            pairs += Hkv * full
        elif not case["causal"]:
            pairs += n * int((kept * size).sum())
        else:
            # (query, key) pairs of each page: queries at or behind the key
            pos = np.arange(np_ * P).reshape(np_, P)
            seen = np.where(pos < L, np.minimum(n, L - pos), 0).sum(1)
            pairs += int((kept * seen).sum())
    return {"bytes": 2 * 2 * keys * D + 2 * 2 * T * Hq * D + 4 * pages,
            "flops": 4 * D * pairs * (Hq // Hkv)}


# ------------------------------------------------------------------ inputs
def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _randn(g, shape, dtype, dev, gain=1.0):
    return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * gain).to(dtype)


def _angles(n, D, dev):
    """cos and sin (n, D/2) in fp32 of the positions 0..n-1, angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, D, 2, device=dev, dtype=torch.float64) / D)
    ang = torch.arange(n, device=dev, dtype=torch.float64)[:, None] * inv[None, :]
    return ang.cos().float(), ang.sin().float()


def _layer(g, case, dt, dev, B, S, values):
    """q, k (and v) as logical (B, H, S, D) views of the memory that the case names."""
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    layout = case.get("layout", "fused")
    heads = [Hq, Hkv] + ([Hkv] if values else [])
    if layout == "heads":
        return [_randn(g, (B, h, S, D), dt, dev, 1.5) for h in heads]
    if layout == "tokens":
        return [_randn(g, (B, S, h, D), dt, dev, 1.5).transpose(1, 2) for h in heads]
    x = _randn(g, (B, S, Hq + 2 * Hkv, D), dt, dev, 1.5)
    parts = (x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:])
    return [p.transpose(1, 2) for p in parts[:len(heads)]]


def _pages(case, ctx, new):
    """Host page table of every request's context and chunk: rows of page numbers, drawn
    without repetition from a pool somewhat larger than needed."""
    P = case["page"]
    need = [-(-(c + n) // P) for c, n in zip(ctx, new)]
    n_pages = sum(need) + 3 + sum(need) // 16
    order = list(range(n_pages))
    random.Random(case["lens"] + 1).shuffle(order)
    rows, at = [], 0
    for m in need:
        rows.append(order[at:at + m])
        at += m
    return rows, n_pages, order[at:]


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]
    st = {"op": op, "case": case}
    if op in ("norm", "norm_back"):
        dt = TYPES[case["dtype"]]
        B, S, D = case["B"], case["S"], case["D"]
        st["q"], st["k"] = _layer(g, case, dt, dev, B, S, False)
        st["qw"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=dev)
        st["kw"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=dev)
        st["cos"], st["sin"] = _angles(S, D, dev)
        if op == "norm_back":
            st["dq"] = _randn(g, (B, case["Hq"], S, D), dt, dev, 0.5)
            st["dk"] = _randn(g, (B, case["Hkv"], S, D), dt, dev, 0.5)
        return st
    ctx, new = _lengths(case)
    T, P, R = sum(new), case["page"], case["R"]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    st["ctx"], st["new"] = ctx, new
    if op == "tables":
        # the pool's order is the seed's: the free list that a user's program holds
        need = [-(-(c + n) // P) for c, n in zip(ctx, new)]
        n_pages = sum(need) + 3 + sum(need) // 16
        order = list(range(n_pages))
        random.Random(seed).shuffle(order)
        table = torch.full((R, max(need)), -1, dtype=torch.int32)
        at = 0
        for r, c in enumerate(ctx):
            have = -(-c // P)
            table[r, :have] = torch.tensor(order[at:at + have], dtype=torch.int32)
            at += have
        st["table"], st["free"], st["n_pages"] = table.to(dev), i32(order[at:]), n_pages
        st["ctx_d"], st["new_d"] = i32(ctx), i32(new)
        return st
    rows, n_pages, _ = _pages(case, ctx, new)
    dt = TYPES[case["dtype"]]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    st["n_pages"] = n_pages
    if op == "append":
        q, k, v = _layer(g, case, dt, dev, 1, T, True)
        st["q"], st["k"], st["v"] = q[0], k[0], v[0]
        st["qw"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=dev)
        st["kw"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=dev)
        st["cos"], st["sin"] = _angles(max(c + n for c, n in zip(ctx, new)), D, dev)
        pos = [c + i for c, n in zip(ctx, new) for i in range(n)]
        slot = [rows[r][(c + i) // P] * P + (c + i) % P
                for r, (c, n) in enumerate(zip(ctx, new)) for i in range(n)]
        st["pos"], st["slots"] = i32(pos), i32(slot)
        st["kc"] = _randn(g, (n_pages, Hkv, P, D), dt, dev)
        st["vc"] = _randn(g, (n_pages, Hkv, P, D), dt, dev)
        return st
    # attention: q in memory by heads, as the pass before it leaves it, long enough for a
    # few keys of thousands to carry much of the weight; what no request holds in the pool
    # is NaN
    st["q"] = _randn(g, (Hq, T, D), dt, dev, 2.5)
    st["kc"] = _randn(g, (n_pages, Hkv, P, D), dt, dev)
    st["vc"] = _randn(g, (n_pages, Hkv, P, D), dt, dev)
    held = torch.zeros(n_pages, dtype=torch.bool)
    for r, (c, n) in enumerate(zip(ctx, new)):
        held[rows[r]] = True
        end = (c + n) % P
        if end:
            st["kc"][rows[r][-1], :, end:] = float("nan")
            st["vc"][rows[r][-1], :, end:] = float("nan")
    spare = (~held).nonzero().flatten().to(dev)
    st["kc"][spare] = float("nan")
    st["vc"][spare] = float("nan")
    width = max(len(x) for x in rows)
    table = torch.full((R, width), -1, dtype=torch.int32)
    for r, x in enumerate(rows):
        table[r, :len(x)] = torch.tensor(x, dtype=torch.int32)
    st["table"] = table.to(dev)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    st["cu_d"], st["ctx_d"], st["max_new"] = i32(cu), i32(ctx), max(new)
    keep = _kept_pages(case)
    st["mask"] = None if keep is None else torch.from_numpy(keep.astype(np.uint8)).to(dev)
    return st


# ------------------------------------------------------------------ plain forms
def _pair_rotate(y, cos, sin, interleaved):
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    h = y.shape[-1] // 2
    a, b = y[..., :h], y[..., h:]
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


def _norm_rotate(x, w, cos, sin, interleaved):
    f = x.float()
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    return _pair_rotate(f * r * w, cos, sin, interleaved).to(x.dtype)


def _norm_rotate_back(x, w, cos, sin, interleaved, dout):
    f = x.float()
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    z = _pair_rotate(dout.float(), cos, -sin, interleaved)
    dw = (z * f * r).sum((0, 1, 2), dtype=torch.float64).float()
    gr = z * w
    dx = r * (gr - f * (r * r) * (gr * f).mean(-1, keepdim=True))
    return dx.to(x.dtype), dw


def _plain_tables(st):
    case, P = st["case"], st["case"]["page"]
    dev = st["table"].device
    c, n = st["ctx_d"].long(), st["new_d"].long()
    T, R = sum(st["new"]), case["R"]
    have = (c + P - 1) // P
    need = (c + n + P - 1) // P - have
    first = need.cumsum(0) - need
    cu = torch.zeros(R + 1, dtype=torch.int32, device=dev)
    cu[1:] = n.cumsum(0)
    table = st["table"]
    col = torch.arange(table.shape[1], device=dev)[None, :]
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    idx = (first[:, None] + col - have[:, None]).clamp(0, max(st["free"].numel() - 1, 0))
    table = torch.where(fresh, st["free"][idx], table)
    req = torch.repeat_interleave(torch.arange(R, device=dev), n, output_size=T)
    pos = torch.arange(T, device=dev) - cu[:-1].long()[req] + c[req]
    slots = table[req, pos // P].long() * P + pos % P
    return {"slots": slots.int(), "positions": pos.int(), "cu": cu, "table": table,
            "taken": need.sum().int().reshape(1)}


def _plain_attend(st):
    case = st["case"]
    Hq, Hkv, P, D = case["Hq"], case["Hkv"], case["page"], case["D"]
    G = Hq // Hkv
    q, kc, vc, out = st["q"], st["kc"], st["vc"], torch.empty_like(st["q"])
    scale = 1.0 / math.sqrt(D)
    at = 0
    for r, (c, n) in enumerate(zip(st["ctx"], st["new"])):
        L = c + n
        pages = st["table"][r, :-(-L // P)].long()
        hide = None
        if case["causal"]:
            hide = (torch.arange(L, device=q.device)[None, :] >
                    torch.arange(c, L, device=q.device)[:, None])
        # as many heads at a time as half a gigabyte of logits holds
        step = max(1, min(Hkv, (1 << 27) // max(G * n * L, 1)))
        for h0 in range(0, Hkv, step):
            h1 = min(Hkv, h0 + step)
            K = kc[pages, h0:h1].transpose(0, 1).reshape(h1 - h0, -1, D)[:, :L].float()
            V = vc[pages, h0:h1].transpose(0, 1).reshape(h1 - h0, -1, D)[:, :L].float()
            Q = q[h0 * G:h1 * G, at:at + n].reshape(h1 - h0, G * n, D).float()
            s = (Q @ K.transpose(1, 2)).mul_(scale).view(h1 - h0, G, n, L)
            if hide is not None:
                s.masked_fill_(hide, -math.inf)
            if st["mask"] is not None:
                m = st["mask"][r, h0:h1, :pages.numel()].bool().repeat_interleave(P, 1)[:, :L]
                s.masked_fill_(~m[:, None, None, :], -math.inf)
            top = s.amax(-1, keepdim=True)
            s.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
            total = s.sum(-1, keepdim=True)
            o = (s.view(h1 - h0, G * n, L) @ V).view(h1 - h0, G, n, D)
            o = torch.where(total > 0, o / total, torch.zeros_like(o))
            out[h0 * G:h1 * G, at:at + n] = o.reshape((h1 - h0) * G, n, D).to(out.dtype)
        at += n
    return out


def _plain(st):
    op, case = st["op"], st["case"]
    if op == "tables":
        return _plain_tables(st)
    if op == "attend":
        return _plain_attend(st)
    inter = case["interleaved"]
    if op == "norm":
        return (_norm_rotate(st["q"], st["qw"], st["cos"], st["sin"], inter).contiguous(),
                _norm_rotate(st["k"], st["kw"], st["cos"], st["sin"], inter).contiguous())
    if op == "norm_back":
        dq, dqw = _norm_rotate_back(st["q"], st["qw"], st["cos"], st["sin"], inter, st["dq"])
        dk, dkw = _norm_rotate_back(st["k"], st["kw"], st["cos"], st["sin"], inter, st["dk"])
        return dq, dk, dqw, dkw
    pos, slots, P = st["pos"].long(), st["slots"].long(), case["page"]
    cos, sin = st["cos"][pos], st["sin"][pos]
    qo = _norm_rotate(st["q"], st["qw"], cos, sin, inter).contiguous()
    ko = _norm_rotate(st["k"], st["kw"], cos, sin, inter)
    st["kc"][slots // P, :, slots % P] = ko.transpose(0, 1)
    st["vc"][slots // P, :, slots % P] = st["v"].transpose(0, 1)
    return qo, st["kc"], st["vc"]


# ------------------------------------------------------------------ the framework's calls
def _own(st):
    import block_sparse_attention_tcgen05_b200 as bsa
    op, case = st["op"], st["case"]
    if op == "tables":
        slots, pos, cu, taken = bsa.paged_block_tables(
            st["ctx_d"], st["new_d"], st["table"], st["free"], sum(st["new"]), case["page"],
            st["n_pages"])
        return {"slots": slots, "positions": pos, "cu": cu, "table": st["table"], "taken": taken}
    if op == "attend":
        return bsa.paged_chunk_attention(st["q"], st["kc"], st["vc"], st["table"], st["cu_d"],
                                         st["ctx_d"], causal=case["causal"], max_new=st["max_new"],
                                         page_mask=st["mask"])
    if op == "norm":
        return bsa.qk_norm_rotation(st["q"], st["k"], st["qw"], st["kw"], st["cos"], st["sin"],
                                    eps=EPS, interleaved=case["interleaved"])
    if op == "norm_back":
        return bsa.qk_norm_rotation_backward(st["dq"], st["dk"], st["q"], st["k"], st["qw"],
                                             st["kw"], st["cos"], st["sin"], eps=EPS,
                                             interleaved=case["interleaved"])
    qo = bsa.paged_qk_norm_append(st["q"], st["k"], st["v"], st["qw"], st["kw"], st["cos"],
                                  st["sin"], st["pos"], st["slots"], st["kc"], st["vc"], eps=EPS,
                                  interleaved=case["interleaved"])
    return qo, st["kc"], st["vc"]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_heads(x, w, cos, sin, interleaved):
    """Normed and rotated rows: the pair as a complex number times exp(i angle)."""
    x = x.double()
    y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w.double()
    D = x.shape[-1]
    if interleaved:
        z = torch.complex(y[..., ::2].contiguous(), y[..., 1::2].contiguous())
    else:
        z = torch.complex(y[..., :D // 2].contiguous(), y[..., D // 2:].contiguous())
    z = z * torch.complex(cos.double(), sin.double())
    if interleaved:
        return torch.view_as_real(z).flatten(-2)
    return torch.cat((z.real, z.imag), -1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "tables":
        # request by request with Python's whole numbers
        P, free = case["page"], st["free"].tolist()
        table, slots, pos, cu, taken = st["table"].tolist(), [], [], [0], 0
        for r, (c, n) in enumerate(zip(st["ctx"], st["new"])):
            for t in range(c, c + n):
                if t // P >= -(-c // P) and (t % P == 0):
                    table[r][t // P] = free[taken]
                    taken += 1
                slots.append(table[r][t // P] * P + t % P)
                pos.append(t)
            cu.append(cu[-1] + n)
        return {k: torch.tensor(x, dtype=torch.int32) for k, x in
                (("slots", slots), ("positions", pos), ("cu", cu), ("table", table),
                 ("taken", [taken]))}
    if op == "norm":
        return tuple(_exact_heads(st[x], st[x + "w"], st["cos"], st["sin"], case["interleaved"])
                     for x in ("q", "k"))
    if op == "norm_back":
        # the chain rule by automatic differentiation of the definition, batch by batch
        dx, dw = [], []
        for x in ("q", "k"):
            w = st[x + "w"].double().requires_grad_()
            parts, total = [], 0
            for b in range(case["B"]):
                for h in range(st[x].shape[1]):
                    a = st[x][b, h].double().requires_grad_()
                    y = _exact_heads(a, w, st["cos"], st["sin"], case["interleaved"])
                    ga, gw = torch.autograd.grad(y, (a, w), st["d" + x][b, h].double())
                    parts.append(ga)
                    total = total + gw
            dx.append(torch.stack(parts).view(case["B"], -1, case["S"], case["D"]))
            dw.append(total)
        return (*dx, *dw)
    if op == "append":
        cos, sin = st["cos"][st["pos"].long()], st["sin"][st["pos"].long()]
        kc, vc = st["kc"].double(), st["vc"].double()
        ko = _exact_heads(st["k"], st["kw"], cos, sin, case["interleaved"])
        P, slots = case["page"], st["slots"].tolist()
        page = torch.tensor([s // P for s in slots], device=kc.device)
        row = torch.tensor([s % P for s in slots], device=kc.device)
        for h in range(case["Hkv"]):
            kc[page, h, row] = ko[h]
            vc[page, h, row] = st["v"][h].double()
        return _exact_heads(st["q"], st["qw"], cos, sin, case["interleaved"]), kc, vc
    # attention, head by head over the list of keys that the request's head keeps
    Hq, Hkv, P, D = case["Hq"], case["Hkv"], case["page"], case["D"]
    dev = st["q"].device
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=dev)
    kept = _kept_pages(case)
    table = st["table"].tolist()
    at = 0
    for r, (c, n) in enumerate(zip(st["ctx"], st["new"])):
        L = c + n
        slots_all = (torch.tensor(table[r][:-(-L // P)], device=dev)[:, None] * P +
                     torch.arange(P, device=dev)[None, :]).flatten()[:L]
        qpos = torch.arange(c, L, device=dev)
        for g in range(Hkv):
            keys = torch.arange(L, device=dev)
            if kept is not None:
                keys = keys[torch.from_numpy(kept[r, g])[keys.cpu() // P].to(dev)]
            if keys.numel() == 0:
                continue
            where = slots_all[keys]
            K = st["kc"][where // P, g, where % P].double()
            V = st["vc"][where // P, g, where % P].double()
            for h in range(g * (Hq // Hkv), (g + 1) * (Hq // Hkv)):
                for i0 in range(0, n, 1024):
                    i1 = min(n, i0 + 1024)
                    e = torch.einsum("id,jd->ij", st["q"][h, at + i0:at + i1].double(), K) / math.sqrt(D)
                    if case["causal"]:
                        e = e + torch.where(keys[None, :] <= qpos[i0:i1, None], 0.0, -math.inf)
                    seen = (e > -math.inf).any(1)
                    p = torch.exp(e - torch.logsumexp(e, 1, keepdim=True))
                    o = torch.einsum("ij,jd->id", p, V)
                    out[h, at + i0:at + i1] = torch.where(seen[:, None], o, torch.zeros_like(o))
        at += n
    return out
