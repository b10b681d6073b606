"""The paged FP8 cache and the two attentions that read it: what is measured, and their plain forms.

The cache holds one latent row per token (K = V = the row): 512 E4M3 values and one fp32 scale, in
pages of a pool that a table [B][max_pages] names.  Three operators work on it:

* csa2_pages_append: RMSNorm, the rotation of the last 64 channels by the token's position, and the
  FP8 quantisation of new rows, written to the page slots of (sequence, position);
* csa2_window_attn: causal attention of 16 heads with a sliding window and a few first tokens that
  stay visible;
* csa2_prefix_attn: attention of a batch over a prefix that all sequences share and each one's own
  tokens, under one softmax.

`own = False`: the plain form, elementary torch operations in 32 bits.  `own = True`: the calls of
sparse_attention_fp4_quant_b200.
"""
import math

import torch

own = False

D, H, ROPE = 512, 16, 64
DEV = "cuda"
SCALE = 1.0 / math.sqrt(D)
EPS = 1e-6


def listed():
    return [
        # the new tokens of one decode step of a batch
        dict(name="append_decode_32", op="append", rows=32, batch=32, ctx=4096, page=64),
        # a ragged step of several prompts' chunks, with unused rows behind them; rows cut out of a wider product
        dict(name="append_ragged_1003", op="append", rows=1003, batch=5, ctx=65519, page=16, pad=37, stride=640),
        # one prefill of a whole prompt
        dict(name="append_prompt_32768", op="append", rows=32768, batch=1, ctx=32768, page=64),
        # one decoded token: the smallest call
        dict(name="window_decode_b1", op="window", batch=1, q=1, ctx=4096, window=128, sink=4, page=64),
        # a decode step of a batch in a sliding-window layer
        dict(name="window_decode_b32", op="window", batch=32, q=1, ctx=131072, window=128, sink=4, page=64),
        # a decode step with a wide window, an odd batch and small pages
        dict(name="window_decode_b61_w4096", op="window", batch=61, q=1, ctx=9001, window=4096, sink=9, page=16),
        # the bounded replay of the last 128 tokens of four sequences: nothing before it is in the cache
        dict(name="window_replay_b4", op="window", batch=4, q=128, ctx=262144, window=128, sink=0, page=64, replay=True),
        # a chunk of a prompt through a sliding-window layer
        dict(name="window_chunk_4096", op="window", batch=1, q=4096, ctx=65536, window=128, sink=4, page=64),
        # chunks of three prompts, one of them shorter, through a wider window
        dict(name="window_chunk_b3_w1024", op="window", batch=3, q=1017, ctx=5003, window=1024, sink=5, page=32),
        # four answers drawn for one prompt
        dict(name="prefix_b4", op="prefix", batch=4, q=1, prefix=4096, ctx=61, page=64),
        # drafts of two tokens checked for each of 21 sequences behind a common document
        dict(name="prefix_b21_q2", op="prefix", batch=21, q=2, prefix=32749, ctx=700, page=16),
        # a batch behind a common context of the longest decode workload
        dict(name="prefix_b32_131k", op="prefix", batch=32, q=1, prefix=131072, ctx=512, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "window", "window", "prefix", "prefix"])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        rows = _log(rng, 1, 32768)
        return dict(op=op, rows=rows, batch=rng.randint(1, min(rows, 32)), ctx=_log(rng, 4096, 262144), page=page,
                    pad=rng.choice([0, rng.randint(1, 40)]), stride=rng.choice([D, D + 8 * rng.randint(1, 64)]))
    if op == "window":
        q = rng.choice([1, 1, rng.randint(2, 4), _log(rng, 5, 4096)])
        window = _log(rng, 1, 4096 if q < 64 else 1024)
        batch = _log(rng, 1, max(1, min(61, 4096 // q)))
        case = dict(op=op, batch=batch, q=q, ctx=_log(rng, q + window, 131072), window=window, sink=rng.randint(0, 16),
                    page=page)
        if rng.random() < 0.2:
            case["replay"], case["sink"] = True, 0
        return case
    q = rng.choice([1, 1, 1, rng.randint(2, 4)])
    batch = _log(rng, 2, 64)
    return dict(op=op, batch=batch, q=q, prefix=_log(rng, 512, max(1024, min(131072, 32 * 131072 // (batch * q)))),
                ctx=_log(rng, q, 1024), page=page)


# ---- inputs ------------------------------------------------------------------------------------

def _lens(case):
    """Tokens of each sequence (the prefix not counted): ctx, a few fewer from sequence to sequence."""
    low = case.get("q", 1)
    return [max(low, case["ctx"] - (b * 61) % max(1, case["ctx"] // 3)) for b in range(case["batch"])]


def _short(case):
    """New tokens of each sequence's chunk: q, and fewer in the last one of a batch of long chunks."""
    q, n = case["q"], [case["q"]] * case["batch"]
    if case["batch"] > 1 and q > 16 and not case.get("replay"):
        n[-1] = q - q // 3
    return n


def _append_counts(case):
    n, B = case["rows"], case["batch"]
    cuts = [n * b // B for b in range(B + 1)]
    counts = [cuts[b + 1] - cuts[b] for b in range(B)]
    return counts


def _latents(n, g):
    x = torch.randn((n, D), device=DEV, generator=g)
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)


def _fill(pool, pool_sc, g):
    """Latent rows in every slot of a pool, as FP8 with a scale per token."""
    flat, sc = pool.view(-1, D), pool_sc.view(-1)
    for r in range(0, flat.shape[0], 1 << 16):
        x = _latents(min(1 << 16, flat.shape[0] - r), g)
        s = x.abs().amax(-1) / 448.0
        flat[r:r + x.shape[0]] = (x / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        sc[r:r + x.shape[0]] = s


def _tables(live, g):
    """Page ids for each sequence's live pages (list of bool lists), -1 for pages not held; pages in random order."""
    width = max(len(r) for r in live)
    flat = torch.tensor([list(r) + [False] * (width - len(r)) for r in live])
    n = int(flat.sum())
    spare = 3
    order = torch.randperm(n + spare, device=DEV, generator=g).cpu()
    table = torch.full(flat.shape, -1, dtype=torch.int32)
    table[flat] = order[:n].to(torch.int32)
    return table.to(DEV), n + spare


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    op, ps = case["op"], case["page"]
    if op == "append":
        counts = _append_counts(case)
        ends = [max(c, n) for c, n in zip(counts, _lens(case))]
        first = [(e - c) // ps for c, e in zip(counts, ends)]
        live = [[False] * f + [True] * (-(-e // ps) - f) for f, e in zip(first, ends)]
        table, n_pages = _tables(live, g)
        pad, n = case.get("pad", 0), case["rows"]
        seq = torch.cat([torch.full((c,), b) for b, c in enumerate(counts)] + [torch.full((pad,), -1)])
        pos = torch.cat([torch.arange(e - c, e) for c, e in zip(counts, ends)] + [torch.zeros(pad, dtype=torch.int64)])
        wide = torch.randn((n + pad, case.get("stride", D)), device=DEV, generator=g) * 1.7
        return dict(op=op, ps=ps, x=wide.to(torch.bfloat16)[:, :D], seq=seq.to(torch.int32).to(DEV),
                    pos=pos.to(torch.int32).to(DEV), norm_w=torch.rand((D,), device=DEV, generator=g) + 0.25,
                    inv_freq=(10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64) / ROPE)).float().to(DEV),
                    pool=torch.zeros((n_pages, ps, D), dtype=torch.uint8, device=DEV),
                    pool_sc=torch.zeros((n_pages, ps), device=DEV), table=table,
                    n_tokens=torch.tensor(ends, dtype=torch.int32, device=DEV))
    B, Q, lens = case["batch"], case["q"], _lens(case)
    state = dict(op=op, ps=ps, pos0=case.get("prefix", 0))
    if op == "window":
        new = _short(case)
        starts = [n - m for n, m in zip(lens, new)] if case.get("replay") else [0] * B
        first = [max(s, n - m - case["window"] + 1, 0) // ps for n, m, s in zip(lens, new, starts)]
        sink_pages = -(-case["sink"] // ps)
        live = [[p < sink_pages or p >= f for p in range(-(-n // ps))] for n, f in zip(lens, first)]
        table, n_pages = _tables(live, g)
        q_pos = torch.full((B, Q), -1, dtype=torch.int32)
        for b in range(B):
            q_pos[b, :new[b]] = torch.arange(lens[b] - new[b], lens[b])
        state.update(window=case["window"], sink=case["sink"],
                     replay=torch.tensor(starts, dtype=torch.int32, device=DEV) if case.get("replay") else None)
    else:
        shared = -(-case["prefix"] // ps)
        live = [[True] * shared] + [[True] * -(-n // ps) for n in lens]
        table, n_pages = _tables(live, g)
        state.update(prefix_table=table[:1, :shared].contiguous(),
                     prefix_tokens=torch.tensor([case["prefix"]], dtype=torch.int32, device=DEV))
        table = table[1:, :max(-(-n // ps) for n in lens)].contiguous()
        q_pos = torch.tensor([[case["prefix"] + n - Q + i for i in range(Q)] for n in lens], dtype=torch.int32)
    pool = torch.empty((n_pages, ps, D), dtype=torch.uint8, device=DEV)
    pool_sc = torch.empty((n_pages, ps), device=DEV)
    _fill(pool, pool_sc, g)
    state.update(pool=pool, pool_sc=pool_sc, table=table, q_pos=q_pos.to(DEV),
                 n_tokens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                 q=torch.randn((B, Q, H, D), device=DEV, generator=g).to(torch.bfloat16))
    return state


# ---- the operators -----------------------------------------------------------------------------

def _own(s):
    import sparse_attention_fp4_quant_b200 as csa
    if "pages" not in s:   # the handles of the caches, which a program keeps beside the tensors
        s["pages"] = csa.Pages.of(s["pool"], s["pool_sc"], s["table"], s["n_tokens"], pos0=s.get("pos0", 0))
        if s["op"] == "prefix":
            s["prefix"] = csa.Pages.of(s["pool"], s["pool_sc"], s["prefix_table"], s["prefix_tokens"])
    if s["op"] == "append":
        csa.csa2_pages_append(s["x"], s["pages"], s["seq"], s["pos"], inv_freq=s["inv_freq"], norm_w=s["norm_w"], eps=EPS)
        return dict(kv=s["pool"].view(torch.float8_e4m3fn), scale=s["pool_sc"])
    if s["op"] == "window":
        out, lse = csa.csa2_window_attn(s["q"], s["pages"], s["q_pos"], window=s["window"], n_sink=s["sink"],
                                        replay_start=s["replay"], sm_scale=SCALE, lse=True)
    else:
        out, lse = csa.csa2_prefix_attn(s["q"], s["prefix"], s["pages"], s["q_pos"], sm_scale=SCALE, lse=True)
    return dict(out=out, lse=lse)


def _rows(s, table, pos, n_tokens):
    """Pool row of each position [B, L] of the sequences of a table, and whether the cache holds it."""
    page = torch.gather(table, 1, (pos // s["ps"]).clamp(0, table.shape[1] - 1).long())
    held = (pos >= 0) & (pos < n_tokens[:, None]) & (pos < table.shape[1] * s["ps"])
    held = held & (page >= 0) & (page < s["pool"].shape[0])
    return torch.where(held, page * s["ps"] + pos.clamp(min=0) % s["ps"], 0).long(), held


def _keys(s, row, held):
    k = s["pool"].view(-1, D)[row].view(torch.float8_e4m3fn).float() * s["pool_sc"].view(-1)[row][..., None]
    return torch.where(held[..., None], k, 0.0)


def _attend(q, keys, visible):
    """q [B, Q, H, D], keys [B, L, D], visible [B, Q, L] -> out bf16, lse: one softmax for each head."""
    B, Q, L = visible.shape
    z = (q.float().reshape(B, Q * H, D) @ keys.transpose(1, 2)).view(B, Q, H, L) * SCALE
    z = torch.where(visible[:, :, None], z, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    out = (p.view(B, Q * H, L) @ keys).view(B, Q, H, D) / torch.where(total > 0, total, 1.0)
    return out.to(torch.bfloat16), (m + torch.log(total)).squeeze(-1)


def run(state):
    s = state
    if own:
        return _own(s)
    if s["op"] == "append":
        x = s["x"].float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["norm_w"]
        angle = s["pos"].double()[:, None] * s["inv_freq"].double()
        c, si = torch.cos(angle).float(), torch.sin(angle).float()
        a, b = y[:, D - ROPE::2], y[:, D - ROPE + 1::2]
        y = torch.cat([y[:, :D - ROPE], torch.stack([a * c - b * si, a * si + b * c], -1).flatten(1)], 1)
        scale = y.abs().amax(-1) / 448.0
        code = (y / torch.where(scale > 0, scale, 1.0)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        seq, n = s["seq"].clamp(min=0).long(), s["pool_sc"].numel()
        row = s["table"][seq, (s["pos"] // s["ps"]).long()] * s["ps"] + s["pos"] % s["ps"]
        source = torch.full((n + 1,), -1, dtype=torch.int64, device=row.device)
        source.scatter_(0, torch.where(s["seq"] >= 0, row, n).long(), torch.arange(row.numel(), device=row.device))
        source, written = source[:n].clamp(min=0), source[:n] >= 0
        pool = torch.where(written[:, None], code[source], s["pool"].view(n, D)).view(s["pool"].shape)
        pool_sc = torch.where(written, scale[source], s["pool_sc"].view(n)).view(s["pool_sc"].shape)
        return dict(kv=pool.view(torch.float8_e4m3fn), scale=pool_sc)
    q_pos, Q = s["q_pos"], s["q_pos"].shape[1]
    if s["op"] == "window":
        w, sink = s["window"], s["sink"]
        last = q_pos.amax(1, keepdim=True)
        first = torch.arange(sink, device=DEV, dtype=torch.int32).expand(q_pos.shape[0], sink)
        near = last - torch.arange(w + Q - 1, device=DEV, dtype=torch.int32)
        pos = torch.cat([first, torch.where(near >= sink, near, -1)], 1)
        row, held = _rows(s, s["table"], pos, s["n_tokens"])
        t, i = pos[:, None], q_pos[:, :, None]
        low = i - w + 1 if s["replay"] is None else torch.maximum(i - w + 1, s["replay"][:, None, None])
        visible = held[:, None] & (t <= i) & ((t >= low) | (t < sink))
        out, lse = _attend(s["q"], _keys(s, row, held), visible)
    else:
        P, B = s["pos0"], q_pos.shape[0]
        row, held = _rows(s, s["prefix_table"], torch.arange(P, device=DEV, dtype=torch.int32)[None], s["prefix_tokens"])
        shared = _keys(s, row, held)[0]
        pos = torch.arange(s["table"].shape[1] * s["ps"], device=DEV, dtype=torch.int32).expand(B, -1)
        row, held = _rows(s, s["table"], pos, s["n_tokens"])
        mine = _keys(s, row, held)
        q = s["q"].float().view(B, Q * H, D)
        z1 = (q.view(B * Q * H, D) @ shared.T).view(B, Q, H, P) * SCALE
        z2 = (q @ mine.transpose(1, 2)).view(B, Q, H, -1) * SCALE
        z2 = torch.where((held[:, None] & (P + pos[:, None] <= q_pos[:, :, None]))[:, :, None], z2, -math.inf)
        m = torch.maximum(z1.amax(-1, keepdim=True), z2.amax(-1, keepdim=True))
        p1, p2 = torch.exp(z1 - m), torch.exp(z2 - m)
        total = p1.sum(-1, keepdim=True) + p2.sum(-1, keepdim=True)
        acc = (p1.view(-1, P) @ shared).view(B, Q, H, D) + (p2.view(B, Q * H, -1) @ mine).view(B, Q, H, D)
        out, lse = (acc / total).to(torch.bfloat16), (m + torch.log(total)).squeeze(-1)
    return dict(out=out, lse=lse)


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    if case["op"] == "append":
        n = case["rows"]
        return {"bytes": n * (2 * D + D + 4 + 8) + case.get("pad", 0) * 4, "flops": n * D * 6}
    lens, B, Q = _lens(case), case["batch"], case["q"]
    rows = B * Q
    moved, pairs = rows * (4 * H * D + 4 * H + 4), 0
    if case["op"] == "window":
        w, sink = case["window"], case["sink"]
        for n, m in zip(lens, _short(case)):
            start = n - m if case.get("replay") else 0
            lo = max(start, n - m - w + 1, 0)
            moved += (n - lo + min(sink, lo)) * (D + 4)
            for i in range(n - m, n):
                low = max(start, i - w + 1, 0)
                pairs += i + 1 - low + min(sink, low)
    else:
        P = case["prefix"]
        moved += (P + sum(lens)) * (D + 4)
        pairs = sum(Q * P + sum(n - Q + 1 + i for i in range(Q)) for n in lens)
    return {"bytes": moved, "flops": pairs * H * D * 4}


# ---- the definition, in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    ps, pool, sc = s["ps"], s["pool"], s["pool_sc"].double()
    if case["op"] == "append":
        kv, scale = pool.view(torch.float8_e4m3fn).double(), sc.clone()
        for b in range(case["batch"]):
            mine = torch.nonzero(s["seq"] == b).flatten()
            if not mine.numel():
                continue
            x, pos = s["x"][mine].double(), s["pos"][mine].long()
            n = x / torch.sqrt(x.square().sum(1, keepdim=True) / D + EPS) * s["norm_w"].double()
            z = torch.complex(n[:, D - ROPE::2].contiguous(), n[:, D - ROPE + 1::2].contiguous())
            turn = pos.double()[:, None] * s["inv_freq"].double()[None]
            n[:, D - ROPE:] = torch.view_as_real(z * torch.polar(torch.ones_like(turn), turn)).flatten(1)
            top = n.abs().max(1).values / 448.0
            page = s["table"][b, pos // ps].long()
            kv[page, pos % ps] = n / top[:, None]
            scale[page, pos % ps] = top
        return dict(kv=kv, scale=scale)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device=DEV)

    def fetch(table, lo, hi):
        t = torch.arange(lo, hi, device=DEV)
        page = table[t // ps].long()
        return pool[page, t % ps].view(torch.float8_e4m3fn).double() * sc[page, t % ps][:, None]

    prefix = fetch(s["prefix_table"][0], 0, case["prefix"]) if case["op"] == "prefix" else None
    for b, n in enumerate(_lens(case)):
        positions = s["q_pos"][b].tolist()
        for c in range(0, case["q"], 64):
            chunk = [p for p in positions[c:c + 64] if p >= 0]
            if not chunk:
                continue
            i = torch.tensor(chunk, device=DEV)[:, None]
            if prefix is None:
                w, sink = case["window"], case["sink"]
                start = n - _short(case)[b] if case.get("replay") else 0
                lo = max(0, start, chunk[0] - w + 1)
                near = fetch(s["table"][b], lo, chunk[-1] + 1)
                few = min(sink, lo)
                keys = torch.cat([fetch(s["table"][b], 0, few), near])
                t = torch.cat([torch.arange(few, device=DEV), torch.arange(lo, chunk[-1] + 1, device=DEV)])[None]
                seen = (t <= i) & ((t > i - w) | (t < sink))
            else:
                keys = torch.cat([prefix, fetch(s["table"][b], 0, n)])
                seen = torch.arange(keys.shape[0], device=DEV)[None] <= i
            z = torch.einsum("qhd,kd->qhk", s["q"][b, c:c + len(chunk)].double(), keys) / math.sqrt(D)
            z = z.masked_fill(~seen[:, None], -math.inf)
            lse[b, c:c + len(chunk)] = torch.logsumexp(z, -1)
            out[b, c:c + len(chunk)] = torch.einsum("qhk,kd->qhd", torch.softmax(z, -1), keys)
    return dict(out=out, lse=lse)
