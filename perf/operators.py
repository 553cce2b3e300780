"""Cases for the operators of the 4-bit key/value cache and of its pages.

Four operators, each as a plain computation in elementary torch operations and
as the library's own calls:

* ``append``: new tokens into a paged 4-bit cache (keys rotated at j mod s and
  rounded to bf16, then every 64 values of a row stored as 4-bit steps of a
  bf16 scale above a bf16 offset), and the stored rows read back as bf16;
* ``decode``: Dual Chunk Attention of one query token per sequence over that
  cache;
* ``remap``: a step of the slots over a pool of pages: slots take over, share,
  cut, grow or drop each other's prefixes, and tails that two slots would both
  write to are copied;
* ``compact``: all pages in use moved to the front of their pools.

The 4-bit pool is uint8 [num_blocks][Hkv][block_rows / 64][tile], one tile
holding 64 keys and values of one head:

    K codes   [64 keys][4 chunks][D/64 groups][2 words][4 bytes]
    K params  [64 keys][D/64]     scale (low 16 bits) and offset, bf16
    V codes   [4][D/64 groups][8 words][16 keys][4 bytes]
    V params  [64 keys][D/64]

Word w of chunk c (K) is word 2 c + w of its group; word i of a group holds its
dimensions 8 i .. 8 i + 7, lowest nibble first.
"""

import math
import random

import numpy as np
import torch

own = False  # set by the caller: run() makes the library's calls where it is true

TILE = 64          # keys of a tile
GROUP = 64         # values that share a scale and an offset


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # one decoded token of each of 16 sequences, written and checked
        dict(name="append_token_b16", op="append", B=16, Hkv=8, D=128, block_rows=128, n_lo=1,
             n_hi=1, t0_lo=1000, t0_hi=9000, s=2048, c=4096),
        # a packed batch of prompts of mixed length, grouped heads
        dict(name="append_prompts_gqa", op="append", B=8, Hkv=8, D=128, block_rows=128, n_lo=512,
             n_hi=8192, t0_lo=0, t0_hi=700, s=2048, c=4096),
        # the next pieces of prompts, as many kv heads as query heads, odd lengths
        dict(name="append_chunks_mha64", op="append", B=5, Hkv=32, D=64, block_rows=64, n_lo=77,
             n_hi=1333, t0_lo=0, t0_hi=5000, s=1000, c=1500),
        # one short chat: latency alone
        dict(name="decode_b1_short", op="decode", B=1, Hq=8, Hkv=1, D=64, block_rows=64, t_lo=900,
             t_hi=1024, s=192, c=256),
        # a batch of chats with as many kv heads as query heads
        dict(name="decode_b24_mha", op="decode", B=24, Hq=32, Hkv=32, D=128, block_rows=64,
             t_lo=17, t_hi=4095, s=2048, c=4096),
        # one document of 100k tokens
        dict(name="decode_b1_100k", op="decode", B=1, Hq=64, Hkv=8, D=128, block_rows=256,
             t_lo=99999, t_hi=100000, s=2048, c=4096),
        # a batch of long contexts
        dict(name="decode_b16_64k", op="decode", B=16, Hq=64, Hkv=8, D=128, block_rows=128,
             t_lo=32768, t_hi=65536, s=2048, c=4096),
        # one step of a beam search over 4-bit pages
        dict(name="remap_beams_kv4", op="remap", kind="kv4", requests=4, width=4, prompt_lo=300,
             prompt_hi=3000, grown_hi=200, block_rows=128, Hkv=8, D=128, layers=4, spare=40),
        # a step of parallel sampling over bf16 pages: many slots, several layers
        dict(name="remap_samples_bf16", op="remap", kind="bf16", requests=16, width=12,
             prompt_lo=500, prompt_hi=4000, grown_hi=600, block_rows=128, Hkv=8, D=128, layers=4,
             spare=200),
        # a few pages to move: latency
        dict(name="compact_small_kv4", op="compact", kind="kv4", slots=12, len_lo=1, len_hi=1500,
             live=0.8, block_rows=64, Hkv=8, D=64, layers=2),
        # a pool half empty after many sequences ended
        dict(name="compact_half_bf16", op="compact", kind="bf16", slots=100, len_lo=500,
             len_hi=4000, live=0.5, block_rows=128, Hkv=8, D=128, layers=2),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], evenly over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "remap", "compact"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 8, 16, 32])
    block_rows = rng.choice([64, 128, 192, 256])
    if op in ("append", "decode"):
        c = _spread(rng, 64, 8000)
        s = rng.randint(max(1, c // 3), c)
    if op == "append":
        B = _spread(rng, 1, 64)
        n_hi = _spread(rng, 1, max(1, min(8192, 32000 * 8 // (B * Hkv))))
        return dict(op=op, B=B, Hkv=Hkv, D=D, block_rows=block_rows,
                    n_lo=rng.randint(1, n_hi), n_hi=n_hi, t0_lo=0, t0_hi=_spread(rng, 1, 9000),
                    s=s, c=c)
    if op == "decode":
        B = _spread(rng, 1, 64)
        t_hi = _spread(rng, 2, max(2, min(120000, 1040000 * 8 // (B * Hkv))))
        return dict(op=op, B=B, Hq=Hkv * rng.choice([1, 2, 4, 5, 8, 12]), Hkv=Hkv, D=D,
                    block_rows=block_rows, t_lo=rng.randint(0, t_hi - 1), t_hi=t_hi, s=s, c=c)
    kind = rng.choice(["kv4", "bf16"])
    layers = rng.randint(1, 4)
    row = (block_rows * Hkv * D * 4) * layers  # bytes of a page over all pools, at most
    if op == "remap":
        requests, width = _spread(rng, 1, 24), rng.randint(1, 12)
        grown = _spread(rng, 1, 600)
        tails = requests * width * (grown // block_rows + 3) * row
        prompt = _spread(rng, 1, 4000)
        if tails > 2.5e9:
            layers, requests = 1, max(1, int(requests * 2.5e9 / tails))
        return dict(op=op, kind=kind, requests=requests, width=width, prompt_lo=1,
                    prompt_hi=prompt, grown_hi=grown, block_rows=block_rows, Hkv=Hkv, D=D,
                    layers=layers, spare=rng.randint(1, 200))
    slots = _spread(rng, 1, 200)
    live = rng.uniform(0.3, 0.95)
    most = max(1.0, 1.8e9 / row * live / slots)
    return dict(op=op, kind=kind, slots=slots, len_lo=0,
                len_hi=max(1, min(_spread(rng, 1, 6000), int(most * block_rows))), live=live,
                block_rows=block_rows, Hkv=Hkv, D=D, layers=layers)


def _lengths(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]: the same work for every seed."""
    return [int(round(lo + (hi - lo) * (i + 0.5) / n)) for i in range(n)]


# ----------------------------------------------------------------------------
# the 4-bit tile, bytes to values and back
# ----------------------------------------------------------------------------
def _tile_bytes(D):
    return 2 * (TILE * D // 2 + TILE * (D // GROUP) * 4)


def _unpack(tiles, D):
    """(codes, scale, offset) of the keys and of the values of uint8 tiles
    [..., tile]: codes uint8 [..., 64, D/64, 64], params fp32 [..., 64, D/64, 1]."""
    lead, gr, nb = tiles.shape[:-1], D // GROUP, TILE * D // 2
    cut = [nb, TILE * gr * 4, nb, TILE * gr * 4]
    kc, kp, vc, vp = torch.split(tiles, cut, dim=-1)
    n = len(lead)
    kc = kc.reshape(*lead, TILE, 4, gr, 2, 4).permute(*range(n), n, n + 2, n + 1, n + 3, n + 4)
    vc = vc.reshape(*lead, 4, gr, 8, 16, 4).permute(*range(n), n, n + 3, n + 1, n + 2, n + 4)
    out = []
    for codes, par in ((kc, kp), (vc, vp)):
        codes = codes.reshape(*lead, TILE, gr, 32)
        codes = torch.stack((codes & 15, codes >> 4), dim=-1).reshape(*lead, TILE, gr, GROUP)
        par = par.contiguous().view(torch.bfloat16).reshape(*lead, TILE, gr, 2).float()
        out.append((codes, par[..., 0:1], par[..., 1:2]))
    return out


def _pack(kc, kp, vc, vp):
    """uint8 tiles [n, tile] of codes [n, 64, gr, 64] and bf16 params [n, 64, gr, 2]."""
    n, gr = kc.shape[0], kc.shape[2]
    kb = (kc[..., 0::2] | (kc[..., 1::2] << 4)).reshape(n, TILE, gr, 4, 2, 4)
    vb = (vc[..., 0::2] | (vc[..., 1::2] << 4)).reshape(n, 4, 16, gr, 8, 4)
    return torch.cat((kb.permute(0, 1, 3, 2, 4, 5).reshape(n, -1),
                      kp.contiguous().view(torch.uint8).reshape(n, -1),
                      vb.permute(0, 1, 3, 4, 2, 5).reshape(n, -1),
                      vp.contiguous().view(torch.uint8).reshape(n, -1)), dim=1)


def _bf16_of(x, up=False):
    """float64 values of `x` rounded once to bf16 (to nearest even, or up)."""
    m, e = torch.frexp(x)
    m = m * 256
    return torch.ldexp(torch.ceil(m) if up else torch.round(m), e - 8)


def _quantised(x):
    """(codes, scale, offset), float64, of bf16 values x [..., 64]: steps of the
    smallest bf16 scale that reaches from the least value to the greatest."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = _bf16_of((hi - lo) / 15, up=True)
    codes = torch.where(scale > 0, torch.round((x - lo) / torch.where(scale > 0, scale, 1)), 0)
    return codes, scale, lo


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _pool_of_values(gen, num_blocks, Hkv, tiles, D):
    """A 4-bit pool of normal keys (some channels stronger than others, as keys
    have them) and values, made a part at a time."""
    pool = torch.empty((num_blocks, Hkv, tiles, _tile_bytes(D)), dtype=torch.uint8, device="cuda")
    flat = pool.view(-1, _tile_bytes(D))
    gr = D // GROUP
    channel = torch.exp(0.4 * _randn(gen, D))
    step = max(1, (1 << 27) // (TILE * D))
    for a in range(0, flat.shape[0], step):
        n = min(step, flat.shape[0] - a)
        got = []
        for weight in (channel, None):
            x = _randn(gen, n, TILE, D)
            x = (x if weight is None else x * weight).bfloat16().float()
            x = x.view(n, TILE, gr, GROUP)
            lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
            scale = (((hi - lo) / 15) * 1.004).bfloat16()
            codes = torch.round((x - lo) / scale.float()).clamp_(0, 15).to(torch.uint8)
            got += [codes, torch.cat((scale, lo.bfloat16()), dim=-1)]
        flat[a:a + n] = _pack(*got)
    return pool


def _tables(case, lens, extra, gen):
    """(block table int32 [B, max_blocks], num_blocks): pages anywhere in the pool."""
    R = case["block_rows"]
    most = max(1, max(-(-n // R) for n in lens))
    num = len(lens) * most + extra
    order = torch.randperm(num, generator=gen, device="cuda", dtype=torch.int64)
    return order[:len(lens) * most].to(torch.int32).view(len(lens), most).contiguous(), num


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if case["op"] in ("remap", "compact"):
        p = _plan(case, seed)
        R, Hkv, D, NB = case["block_rows"], case["Hkv"], case["D"], p["num_blocks"]
        if case["kind"] == "kv4":
            shape = (case["layers"], NB, Hkv, R // TILE, _tile_bytes(D))
            pools = torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.uint8)
        else:
            pools = torch.empty((2 * case["layers"], NB, R, Hkv, D), dtype=torch.bfloat16,
                                device="cuda")
            pools.normal_(generator=gen)
        st = {"pools": pools, **{k: ints(v) for k, v in p.items() if k != "num_blocks"}}
        return {"case": dict(case), **st}
    B, Hkv, D, R = case["B"], case["Hkv"], case["D"], case["block_rows"]
    rng = random.Random(seed)
    if case["op"] == "append":
        n, t0 = (_lengths(case[k + "_lo"], case[k + "_hi"], B) for k in ("n", "t0"))
        rng.shuffle(n)
        rng.shuffle(t0)
        cu = np.concatenate(([0], np.cumsum(n))).tolist()
        table, num = _tables(case, [a + b for a, b in zip(t0, n)], 3, gen)
        pool = torch.zeros((num, Hkv, R // TILE, _tile_bytes(D)), dtype=torch.uint8, device="cuda")
        k = (_randn(gen, cu[-1], Hkv, D) * torch.exp(0.4 * _randn(gen, D))).bfloat16()
        v = _randn(gen, cu[-1], Hkv, D).bfloat16()
        return {"case": dict(case), "k": k, "v": v, "pool": pool, "table": table, "cu": ints(cu),
                "t0": ints(t0)}
    t = _lengths(case["t_lo"], case["t_hi"] - 1, B)
    rng.shuffle(t)
    table, num = _tables(case, [x + 1 for x in t], 3, gen)
    q = _randn(gen, B, case["Hq"], D).bfloat16()
    return {"case": dict(case), "q": q, "pool": _pool_of_values(gen, num, Hkv, R // TILE, D),
            "table": table, "t": ints(t)}


def _plan(case, seed):
    """Slots, lengths, tables and reference counts of a pool in use (plain
    lists); what a scheduler has decided for the next step."""
    rng = random.Random(seed)
    R = case["block_rows"]
    pages = lambda n: -(-n // R)  # noqa: E731
    rows, lens, src, new = [], [], [], []
    count = 0  # pages named 0, 1, .. first and shuffled at the end
    if case["op"] == "remap":
        prompts = _lengths(case["prompt_lo"], case["prompt_hi"], case["requests"])
        grown = _lengths(0, case["grown_hi"], case["requests"])
        random.Random(0).shuffle(grown)  # the same pairs, and sizes, for every seed
        for r, (prompt, g) in enumerate(zip(prompts, grown)):
            shared = list(range(count, count + prompt // R))
            count += len(shared)
            ends = r % 8 == 7  # this request is done; another one takes its slots
            for w in range(case["width"]):
                mine = pages(prompt + g) - len(shared)
                rows.append(shared + list(range(count, count + mine)))
                count += mine
                lens.append(prompt + g)
                src.append(-1 if ends else r * case["width"] + rng.randrange(case["width"]))
                new.append(max(1, prompt // 2) if ends else prompt + g + 1)
        num = count + case["spare"] + sum(
            pages(n) if f < 0 else 1 + pages(n) - pages(m) for n, m, f in zip(new, lens, src))
    else:
        lens = _lengths(case["len_lo"], case["len_hi"], case["slots"])
        rng.shuffle(lens)
        for n in lens:
            mine = pages(n)
            rows.append(list(range(count, count + mine)))
            count += mine
        num = max(1, int(count / case["live"]))
    most = max(1, max([len(r) for r in rows] + [pages(n) for n in new]))
    at = list(range(num))
    rng.shuffle(at)
    refs = [0] * num
    table = []
    for r in rows:
        for p in r:
            refs[at[p]] += 1
        table.append([at[p] for p in r] + [-1] * (most - len(r)))
    got = {"table": table, "refs": refs, "lens": lens, "num_blocks": num}
    return {**got, "src": src, "new": new} if case["op"] == "remap" else got


# ----------------------------------------------------------------------------
# the operators
# ----------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "decode": _own_decode, "remap": _own_remap,
                "compact": _own_compact}[op](state)
    return {"append": _plain_append, "decode": _plain_decode, "remap": _plain_remap,
            "compact": _plain_compact}[op](state)


def _own_append(st):
    import long_context_attention_dca_b200 as dca
    c = st["case"]
    dca.dca_kv4_append_paged(st["k"], st["v"], st["pool"], st["table"], st["cu"], st["t0"],
                             c["s"], c["c"])
    return dca.dca_kv4_read_paged(st["pool"], st["table"], st["cu"], st["t0"],
                                  st["k"].shape[0], c["D"])


def _own_decode(st):
    import long_context_attention_dca_b200 as dca
    c = st["case"]
    return dca.dca_attn_decode_kv4_paged(st["q"], st["pool"], st["table"], st["t"], c["s"], c["c"])


def _own_remap(st):
    import long_context_attention_dca_b200 as dca
    table, refs, info = dca.dca_pages_remap(st["src"], st["lens"], st["new"], st["table"],
                                            st["refs"], st["pools"], st["case"]["block_rows"])
    return table, refs, info, _whole(st["pools"])


def _own_compact(st):
    import long_context_attention_dca_b200 as dca
    table, refs, moved, info = dca.dca_pages_compact(st["lens"], st["table"], st["refs"],
                                                     st["pools"], st["case"]["block_rows"])
    return table, refs, moved, info, _whole(st["pools"])


def _whole(pools):
    """A pool's contents as whole numbers: pages are moved bit for bit."""
    return pools if pools.dtype == torch.uint8 else pools.view(torch.int16)


def _angles(pos, D):
    """pos [...] -> angles [..., D/2] in 64 bits."""
    k = torch.arange(D // 2, device=pos.device, dtype=torch.float64)
    return pos.double()[..., None] * torch.pow(10000.0, -2.0 * k / D)


def _plain_append(st):
    case = st["case"]
    D, h = case["D"], case["D"] // 2
    row = torch.arange(st["k"].shape[0], device=st["k"].device)
    seq = torch.searchsorted(st["cu"][1:].contiguous(), row.to(torch.int32), right=True)
    pos = (st["t0"][seq] + row - st["cu"][seq]) % case["s"]
    a = _angles(pos, D)[:, None, :]
    # in 64 bits: a value next to a rounding border decides a whole step
    x, co, si = st["k"].double(), torch.cos(a), torch.sin(a)
    key = _bf16_of(torch.cat((x[..., :h] * co - x[..., h:] * si,
                              x[..., h:] * co + x[..., :h] * si), dim=-1))
    out = []
    for y in (key, st["v"].double()):
        codes, scale, lo = _quantised(y.view(*y.shape[:-1], D // GROUP, GROUP))
        out.append((codes * scale + lo).reshape(y.shape).to(torch.bfloat16))
    return tuple(out)


def _plain_decode(st):
    case = st["case"]
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    s, c, h = case["s"], case["c"], D // 2
    t = st["t"].long()
    tiles = st["pool"][st["table"].long()]  # [B, blocks, Hkv, tiles, bytes]
    tiles = tiles.permute(0, 2, 1, 3, 4)
    (kc, ks, ko), (vc, vs, vo) = _unpack(tiles, D)
    key = (kc * ks + ko).reshape(B, Hkv, -1, D)
    del kc
    # the query at its three positions
    im = t % s
    pos = torch.stack((im, torch.where(im < c - s, s + im, c - 1),
                       torch.full_like(im, c - 1)), dim=1)
    a = _angles(pos, D)
    co, si = torch.cos(a).float()[:, :, None], torch.sin(a).float()[:, :, None]
    x = st["q"].float()[:, None]
    q = torch.cat((x[..., :h] * co - x[..., h:] * si, x[..., h:] * co + x[..., :h] * si), dim=-1)
    q = q.view(B, 3, Hkv, Hq // Hkv, D).transpose(1, 2) * (1.0 / math.sqrt(D))
    score = torch.matmul(q.reshape(B, Hkv, -1, D), key.transpose(2, 3))
    del key
    score = score.view(B, Hkv, 3, Hq // Hkv, -1)
    j = torch.arange(score.shape[-1], device=t.device)
    gap = ((t // s)[:, None] - j // s)[:, None, None, :]
    score = torch.where(gap == 0, score[:, :, 0],
                        torch.where(gap == 1, score[:, :, 1], score[:, :, 2]))
    score = score.masked_fill((j > t[:, None])[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    val = (vc * vs + vo).reshape(B, Hkv, -1, D)
    del vc
    out = torch.matmul(p, val) / total
    lse = (top + torch.log(total)).view(B, Hq)
    return out.reshape(B, Hq, D).to(torch.bfloat16), lse


def _pages_of(n, R):
    return (n + R - 1) // R


def _units(pools, kind):
    """Pools as [n, num_blocks, outer, units, unit]: the rows of a page in units
    that are copied whole (bf16: one row; 4 bits: a tile of 64 rows of a head)."""
    if kind == "kv4":
        return pools, TILE
    n, num, R = pools.shape[:3]
    return pools.view(n, num, 1, R, -1), 1


def _plain_remap(st):
    R = st["case"]["block_rows"]
    table, refs = st["table"].long(), st["refs"].long()
    src, old, new = st["src"].long(), st["lens"].long(), st["new"].long()
    B, most, num = table.shape[0], table.shape[1], refs.shape[0]
    p = torch.arange(most, device=table.device)
    slot = torch.arange(B, device=table.device)
    none = torch.full((), num, device=table.device)  # a place of its own for "no page"
    count = torch.cat((refs, refs.new_zeros(1)))
    one = torch.ones_like(table)
    used = p < _pages_of(old, R)[:, None]
    count = count.index_add(0, torch.where(used, table, none).flatten(), -one.flatten())
    keep = torch.where(src >= 0, torch.minimum(old[src.clamp(min=0)], new), 0)
    full, rest = keep // R, keep % R
    rows = table[src.clamp(min=0)]
    shared = p < full[:, None]
    count = count.index_add(0, torch.where(shared, rows, none).flatten(), one.flatten())
    tail = rows.gather(1, full.clamp(max=most - 1)[:, None])[:, 0]
    tail = torch.where(rest > 0, tail, none)
    first = torch.full((num + 1,), B, device=table.device).scatter_reduce(0, tail, slot, "amin")
    stays = (rest > 0) & (count[tail] == 0) & (first[tail] == slot)
    count = count.index_add(0, torch.where(stays, tail, none), one[:, 0])
    # free pages, lowest first; the slots take theirs in order
    free = torch.argsort((count[:num] != 0).to(torch.int8), stable=True)
    begin = full + stays
    need = _pages_of(new, R) - begin
    start = torch.cumsum(need, 0) - need
    fresh = (p >= begin[:, None]) & (p < _pages_of(new, R)[:, None])
    at = (start[:, None] + p - begin[:, None]).clamp(0, num - 1)
    out = torch.where(fresh, free[at], torch.where(p < begin[:, None], rows, -1))
    count = count.index_add(0, torch.where(fresh, free[at], none).flatten(), one.flatten())
    copies = ((rest > 0) & ~stays).nonzero()[:, 0]
    units, rows_of = _units(st["pools"], st["case"]["kind"])
    a, b = tail[copies], out[copies].gather(1, full[copies][:, None])[:, 0]
    whole = _pages_of(rest[copies], rows_of)
    taken = torch.arange(units.shape[3], device=table.device) < whole[:, None]
    taken = taken[None, :, None, :, None]
    units[:, b] = torch.where(taken, units[:, a], units[:, b])
    left = (count[:num] == 0).sum()
    info = torch.stack((left, (~stays & (rest > 0)).sum())).to(torch.int32)
    return out.to(torch.int32), count[:num].to(torch.int32), info, _whole(st["pools"])


def _plain_compact(st):
    R = st["case"]["block_rows"]
    table, refs = st["table"].long(), st["refs"]
    num = refs.shape[0]
    page = torch.arange(num, device=table.device)
    live = refs > 0
    n = live.sum()
    hole, late = ~live & (page < n), live & (page >= n)
    holes = torch.argsort((~hole).to(torch.int8), stable=True)
    rank = torch.cumsum(late, 0) - 1
    to = torch.where(late, holes[rank.clamp(min=0)], torch.where(live, page, -1))
    back = torch.where(live, to, num)
    out_refs = torch.zeros(num + 1, dtype=torch.int32, device=table.device)
    out_refs = out_refs.scatter(0, back, refs)[:num]
    out_refs = torch.where(page < n, out_refs, 0)
    used = torch.arange(table.shape[1], device=table.device) < _pages_of(st["lens"], R)[:, None]
    out = torch.where(used, to[torch.where(used, table, 0)], -1)
    a = late.nonzero()[:, 0]
    st["pools"][:, to[a]] = st["pools"][:, a]
    info = torch.stack((n, late.sum())).to(torch.int32)
    return (out.to(torch.int32), out_refs, to.to(torch.int32), info, _whole(st["pools"]))


# ----------------------------------------------------------------------------
# work
# ----------------------------------------------------------------------------
def work(case):
    if case["op"] in ("append", "decode"):
        D, Hkv = case["D"], case["Hkv"]
        stored = Hkv * (D + D // GROUP * 8)  # a token's bytes in the cache
    if case["op"] == "append":
        T = sum(_lengths(case["n_lo"], case["n_hi"], case["B"]))
        return {"bytes": T * (stored + 2 * Hkv * D * 4), "flops": T * Hkv * D * 16}
    if case["op"] == "decode":
        t = _lengths(case["t_lo"], case["t_hi"] - 1, case["B"])
        keys = sum(x + 1 for x in t)
        rows = case["B"] * case["Hq"]
        return {"bytes": keys * stored + rows * (D * 4 + 4), "flops": 4 * D * case["Hq"] * keys}
    p = _plan(case, 0)
    R, Hkv, D = case["block_rows"], case["Hkv"], case["D"]
    pools = case["layers"] * (1 if case["kind"] == "kv4" else 2)
    unit, outer, unit_rows = (_tile_bytes(D), Hkv, TILE) if case["kind"] == "kv4" else (
        Hkv * D * 2, 1, 1)
    lists = 8 * len(p["table"]) * len(p["table"][0]) + 8 * len(p["refs"])
    if case["op"] == "compact":
        n = sum(r > 0 for r in p["refs"])
        units = sum(r > 0 for r in p["refs"][n:]) * (R // unit_rows)
    else:
        units = sum(-(-rows // unit_rows) for _, _, rows in _remap_copies(p, R)[3])
    return {"bytes": lists + 2 * units * outer * unit * pools, "flops": 0}


# ----------------------------------------------------------------------------
# the definitions once more, in 64 bits and step by step
# ----------------------------------------------------------------------------
def _remap_copies(p, R):
    """The step of the slots as a scheduler would do it one slot at a time:
    (table, refs, pages left, [(from, to, rows)])."""
    refs = list(p["refs"])
    most = len(p["table"][0])
    for row, n in zip(p["table"], p["lens"]):
        for page in row[:-(-n // R)]:
            refs[page] -= 1
    kept = []
    for f, n in zip(p["src"], p["new"]):
        keep = 0 if f < 0 else min(p["lens"][f], n)
        kept.append((keep // R, keep % R))
        for page in p["table"][f][:keep // R]:
            refs[page] += 1
    owner = [False] * len(kept)
    taken = set(i for i, r in enumerate(refs) if r > 0)
    for b, (full, rest) in enumerate(kept):
        if rest and p["table"][p["src"][b]][full] not in taken:
            owner[b] = True
            taken.add(p["table"][p["src"][b]][full])
    for b, mine in enumerate(owner):
        if mine:
            refs[p["table"][p["src"][b]][kept[b][0]]] = 1
    free = iter([i for i, r in enumerate(refs) if r == 0])
    table, copies = [], []
    for b, (full, rest) in enumerate(kept):
        row = list(p["table"][p["src"][b]][:full + owner[b]]) if full or rest else []
        while len(row) < -(-p["new"][b] // R):
            page = next(free)
            refs[page] = 1
            if len(row) == full and rest:
                copies.append((p["table"][p["src"][b]][full], page, rest))
            row.append(page)
        table.append(row + [-1] * (most - len(row)))
    return table, refs, sum(r == 0 for r in refs), copies


def _codes64(tiles, D, what):
    """Values (float64 [n, 64, D]) of byte tiles [n, tile], found by their places."""
    gr = D // GROUP
    key, d = np.meshgrid(np.arange(TILE), np.arange(D), indexing="ij")
    g, i, nib = d // 64, (d % 64) // 8, d % 8
    if what == "k":
        word = (key * 4 + i // 2) * gr * 2 + g * 2 + i % 2
        first, par = 0, TILE * D // 2
    else:
        word = ((key // 16 * gr + g) * 8 + i) * 16 + key % 16
        first = TILE * D // 2 + TILE * gr * 4
        par = first + TILE * D // 2
    place = torch.from_numpy(first + word * 4 + nib // 2).to(tiles.device)
    shift = torch.from_numpy(nib % 2 * 4).to(tiles.device)
    code = ((tiles[:, place].int() >> shift) & 15).double()
    at = torch.from_numpy(par + (key * gr + g) * 4).to(tiles.device)
    half = lambda o: ((tiles[:, at + o + 1].int() << 24) | (  # noqa: E731
        tiles[:, at + o].int() << 16)).view(torch.float32).double()
    return code * half(0) + half(2)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, st)
    if case["op"] == "decode":
        return _exact_decode(case, st)
    return None  # pages are moved, nothing is computed


def _exact_append(case, st):
    D, h, s = case["D"], case["D"] // 2, case["s"]
    cu, t0 = st["cu"].tolist(), st["t0"].tolist()
    theta = torch.tensor([10000.0 ** (-2.0 * k / D) for k in range(h)], dtype=torch.float64)
    keys = []
    for b in range(case["B"]):
        pos = (torch.arange(t0[b], t0[b] + cu[b + 1] - cu[b]) % s).double()
        turn = torch.polar(torch.ones((), dtype=torch.float64), pos[:, None] * theta).cuda()
        x = st["k"][cu[b]:cu[b + 1]].double()
        z = torch.complex(x[..., :h].contiguous(), x[..., h:].contiguous()) * turn[:, None, :]
        keys.append(torch.cat((z.real, z.imag), dim=-1))
    key = torch.cat(keys)
    power = torch.exp2(torch.floor(torch.log2(key.abs())) - 7)  # of the last bf16 place
    key = torch.where(key == 0, key, torch.round(key / power) * power)
    out = []
    for y in (key, st["v"].double()):
        y = y.reshape(-1, GROUP)
        lo, hi = torch.aminmax(y, dim=1)
        step = (hi - lo) / 15
        place = torch.exp2(torch.floor(torch.log2(step.clamp(min=1e-300))) - 7)
        step = torch.ceil(step / place) * place
        code = torch.round((y - lo[:, None]) / step[:, None].clamp(min=1e-300))
        out.append((lo[:, None] + code * step[:, None]).view(key.shape))
    return tuple(out)


def _exact_decode(case, st):
    Hq, Hkv, D, R = case["Hq"], case["Hkv"], case["D"], case["block_rows"]
    s, c, h, G = case["s"], case["c"], D // 2, Hq // Hkv
    theta = torch.tensor([10000.0 ** (-2.0 * k / D) for k in range(h)], dtype=torch.float64)
    outs, lses = [], []
    for b, t in enumerate(st["t"].tolist()):
        n, ci, im = t + 1, t // s, t % s
        blocks = st["table"][b, :-(-n // R)].long()
        pos = torch.tensor([im, s + im if im < c - s else c - 1, c - 1], dtype=torch.float64)
        turn = torch.polar(torch.ones((), dtype=torch.float64), pos[:, None] * theta).cuda()
        x = st["q"][b].double()
        z = torch.complex(x[:, :h].contiguous(), x[:, h:].contiguous())[None] * turn[:, None, :]
        q = torch.cat((z.real, z.imag), dim=-1) / math.sqrt(D)  # [3, Hq, D]
        piece = (ci - torch.arange(n, device="cuda") // s).clamp(max=2)
        for g in range(Hkv):
            tiles = st["pool"][blocks, g].reshape(-1, _tile_bytes(D))
            key = _codes64(tiles, D, "k").view(-1, D)[:n]
            score = torch.einsum("phd,jd->phj", q[:, g * G:(g + 1) * G], key)
            score = score.gather(0, piece[None, None].expand(1, G, n))[0]
            lse = torch.logsumexp(score, dim=1)
            val = _codes64(tiles, D, "v").view(-1, D)[:n]
            outs.append(torch.exp(score - lse[:, None]) @ val)
            lses.append(lse)
    B = case["B"]
    return torch.stack(outs).view(B, Hq, D), torch.stack(lses).view(B, Hq)
