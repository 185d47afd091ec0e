"""The paged 8-bit cache's operators, as they are measured.

Three kinds of case, each one pass through one operator:

- "append": rotate the new tokens' keys, quantise keys and values to e4m3 with one power-of-two
  scale for each (page, KV head), and write them into the sequences' pages;
- "token": attention of one new token of each sequence over its paged cache (serving);
- "prompt": causal attention of many new tokens of each sequence over its paged cache (prompts,
  chunks of prompts, several requests of different lengths at once).

A pool is [n_pages][n_kv_heads][page][head_dim] e4m3 codes with scales [n_pages][n_kv_heads]; a
code stands for code * scale.  Sequence b has lens[b] tokens in the cache, the last news[b] of
them new in this pass.

`run` computes the plain form (elementary torch operations in 32 bits, angles in 64) where `own`
is false, and calls the framework's entry points where it is true.  `exact` is the definition in
64 bits, one sequence and head at a time.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -100  # exponent of the scale of a page that holds only zeros


def _case(name, kind, dtype, hq, hkv, d, page, lens, news, base=10000.0, window=0):
    return {"name": name, "kind": kind, "dtype": dtype, "hq": hq, "hkv": hkv, "d": d, "page": page,
            "lens": ",".join(map(str, lens)), "news": ",".join(map(str, news)), "base": base,
            "window": window}


def listed():
    # serving batch with odd lengths, an empty slot (a padded batch) and sequences of one token
    serve = [((b * 2654435761) % 4093) + 1 for b in range(61)] + [1, 0, 4097]
    # requests of one step of a chunked scheduler: a whole prompt, chunks, single tokens
    mixed_len = [1024, 4099, 37, 2011, 7777, 513, 1, 3000]
    mixed_new = [1024, 1023, 37, 512, 1, 513, 1, 333]
    # prompts of a batch admitted at once, odd lengths
    admitted = [8192, 4001, 2048, 1023, 517, 333, 64, 206]
    return [
        # one decode step's append at the smallest batch: launch latency
        _case("append_token_b4", "append", "bf16", 32, 8, 128, 64, [32768, 32001, 17, 1], [1] * 4),
        # one decode step's append of a serving batch, multi-head keys
        _case("append_token_b64_mha", "append", "bf16", 32, 32, 128, 16, [n + 5 for n in serve],
              [1] * 64),
        # prompts of several requests written at once, behind what is there already
        _case("append_prompt_16k", "append", "bf16", 32, 8, 128, 16, [n + 41 for n in admitted],
              admitted),
        # the same in 32 bits, small heads, largest pages
        _case("append_prompt_f32", "append", "f32", 16, 4, 64, 128, [4099, 2500], [4099, 1777]),
        # LLaMA2-7B-shaped decode step, one sequence of 4K: the smallest attention
        _case("token_4k_mha_b1", "token", "bf16", 32, 32, 128, 16, [4096], [1]),
        # Mistral-7B-shaped decode step, four sequences of 32K
        _case("token_32k_b4", "token", "bf16", 32, 8, 128, 64, [32768] * 4, [1] * 4),
        # LLaMA3.1-8B-shaped decode step, ragged 16K to 128K: the largest single-token case
        _case("token_128k_ragged", "token", "bf16", 32, 8, 128, 128, [16384, 32768, 65536, 131072],
              [1] * 4, 500000.0),
        # a serving batch of 64 short sequences of odd lengths, one of them an empty slot
        _case("token_serve_b64", "token", "bf16", 32, 8, 128, 16, serve, [1] * 64),
        # 32-bit storage, small heads, groups of two
        _case("token_8k_f32", "token", "f32", 8, 4, 64, 32, [8191, 1000, 5003], [1] * 3),
        # a whole prompt of 4K
        _case("prompt_4k", "prompt", "bf16", 32, 8, 128, 64, [4096], [4096]),
        # one step of a scheduler that mixes prompts, chunks and single tokens
        _case("prompt_mixed", "prompt", "bf16", 32, 8, 128, 16, mixed_len, mixed_new),
        # a chunk of 2K tokens at the end of a 32K context: the largest work
        _case("prompt_chunk_32k", "prompt", "bf16", 32, 8, 128, 128, [32768], [2048], 500000.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["append", "token", "prompt"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    hq, hkv = rng.choice([(32, 8), (32, 8), (32, 32), (16, 2), (8, 4), (4, 4), (8, 1)])
    base = rng.choice([10000.0, 500000.0])
    window = rng.choice([0, 0, 0, _log_int(rng, 1, 8192)])
    batch = _log_int(rng, 1, 64 if kind != "prompt" else 8)
    top = _log_int(rng, 1, {"append": 16384, "token": 131072, "prompt": 32768}[kind])
    lens = [top] + [_log_int(rng, 1, top) for _ in range(batch - 1)]
    if rng.random() < 0.25:
        lens[-1] = 0  # an empty slot of a padded batch
    if kind == "token":
        news = [1] * batch
    else:
        most = _log_int(rng, 1, 2048 if kind == "prompt" else 8192)
        news = [min(n, _log_int(rng, 1, most)) for n in lens]
    cap = work(listed()[6]), work(listed()[11])
    while True:
        c = _case("", kind, dtype, hq, hkv, d, page, lens, news, base, window)
        del c["name"]
        w = work(c)
        padded = 4.0 * batch * hq * max(news) * max(lens)  # the plain form's largest intermediate
        held = 8.0 * batch * hkv * max(lens) * d           # and its keys and values
        flops = cap[1]["flops"] * (1.0 if dtype == "bf16" else 0.1)
        if (w["bytes"] <= cap[0]["bytes"] and w["flops"] <= flops and padded <= 8.6e9
                and held <= 1.6e10):
            return c
        lens = [n * 3 // 4 for n in lens]
        news = [min(n, max(1, m * 3 // 4)) if kind != "token" else 1 for n, m in zip(lens, news)]


def _ints(text):
    return [int(x) for x in text.split(",")]


def _pairs(n, m, window):
    """Query-key pairs of m queries at the end of n tokens."""
    first = n - m
    total = 0
    for i in range(max(0, first), n):
        total += min(i + 1, window) if window else i + 1
    return total


def work(case):
    lens, news = _ints(case["lens"]), _ints(case["news"])
    e = 2 if case["dtype"] == "bf16" else 4
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    new = sum(min(n, m) for n, m in zip(lens, news))
    if case["kind"] == "append":
        # keys and values in, codes out, the touched pages' scales
        pages = sum(-(-n // page) - (n - min(n, m)) // page for n, m in zip(lens, news))
        return {"bytes": 2 * hkv * (new * d * (e + 1) + pages * 4), "flops": 3.0 * new * hkv * d}
    # queries in, outputs out, every key and value code that a query sees once, and their scales
    w = case["window"]
    seen = sum((min(n, w + min(n, m) - 1) if w else n) for n, m in zip(lens, news) if m)
    pairs = sum(_pairs(n, m, w) for n, m in zip(lens, news))
    return {"bytes": 2 * new * hq * d * e + 2 * hkv * seen * (d + 4.0 / page),
            "flops": 4.0 * pairs * hq * d}


def _exponent(amax):
    """The least e with amax <= 448 * 2^e (MIN_EXP for zeros)."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)


def _scale_of(amax):
    return torch.ldexp(torch.ones_like(amax), _exponent(amax))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    lens, news = _ints(case["lens"]), _ints(case["news"])
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    batch = len(lens)
    held = [-(-n // page) for n in lens]
    n_pages, max_pages = sum(held) + 3, max(held) + 1
    order = torch.randperm(n_pages, generator=g, device=dev).tolist()
    table = np.full((batch, max_pages), -1, np.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    offsets = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    n_tokens = int(offsets[-1])

    def rand(*shape):
        return torch.randn(shape, generator=g, device=dev)

    # channels of different strength, as keys have
    gain = torch.exp(0.4 * rand(hkv, 1, d // 2)).repeat(1, 1, 2)
    gain = gain / gain.square().mean().sqrt()
    s = {"case": case, "page_table": torch.from_numpy(table).to(dev),
         "seq_lens": torch.tensor(lens, dtype=torch.int32, device=dev),
         "q_offsets": torch.from_numpy(offsets).to(dev),
         "seq_lens_host": lens, "news_host": news, "offsets_host": offsets.tolist()}
    for name in ("k", "v"):
        x = rand(n_pages, hkv, page, d)
        if name == "k":
            x = x * gain
        sc = _scale_of(x.abs().amax((2, 3)))
        s[name + "_pages"] = (x / sc[:, :, None, None]).to(torch.float8_e4m3fn)
        s[name + "_scales"] = sc
        del x
    if case["kind"] == "append":
        s["K_new"] = (rand(n_tokens, hkv, d) * gain[:, 0]).to(dt)
        s["V_new"] = rand(n_tokens, hkv, d).to(dt)
    else:
        s["q"] = (1.5 * rand(n_tokens, hq, d)).to(dt)
        s["out"] = torch.zeros(n_tokens, hq, d, dtype=dt, device=dev)
    if own:
        from latent_space_sparse_b200 import salsc
        s["cache"] = salsc.PagedCache(
            hq, hkv, d, page, n_pages, s["page_table"], s["seq_lens"],
            None if case["kind"] == "token" else s["q_offsets"],
            n_tokens=n_tokens, max_q=max(news), rope_base=case["base"], window=case["window"],
            dtype=dt)
    return s


def _tokens(s):
    """Sequence, index in the sequence's new tokens, and cache position of every new token."""
    offs = s["q_offsets"].long()
    count = offs[1:] - offs[:-1]
    n = s["offsets_host"][-1]
    b = torch.repeat_interleave(torch.arange(count.numel(), device=offs.device), count,
                                output_size=n)
    i = torch.arange(n, device=offs.device) - offs[b]
    return b, i, s["seq_lens"].long()[b] - count[b] + i


def _rotate(x, pos, base):
    """Rotate-half position rotation of x [n][heads][d] at pos [n]; angles in 64 bits."""
    half = x.shape[-1] // 2
    theta = base ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    ang = pos.double()[:, None] * theta
    c, sn = ang.cos().float()[:, None], ang.sin().float()[:, None]
    x = x.float()
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * sn, b * c + a * sn], -1)


def _append_plain(s):
    case = s["case"]
    page, d = case["page"], case["d"]
    b, i, pos = _tokens(s)
    keep = torch.arange(b.numel(), device=b.device)[pos >= 0] if min(
        n - m for n, m in zip(s["seq_lens_host"], s["news_host"])) < 0 else slice(None)
    b, pos = b[keep], pos[keep]
    pg, slot = s["page_table"].long()[b, pos // page], pos % page
    # the sequences with new tokens, their first touched page and first new slot
    lens = s["seq_lens"].long()
    offs = s["q_offsets"].long()
    count = torch.minimum(offs[1:] - offs[:-1], lens)
    start = lens - count
    first = s["page_table"].long().gather(1, (start // page)[:, None])[:, 0]
    live = (count > 0) & (first >= 0)
    spare = first.new_full((), s["k_pages"].shape[0])  # writes of idle sequences go nowhere
    for name in ("k", "v"):
        x = s["K_new" if name == "k" else "V_new"][keep].float()
        if name == "k":
            amax = (x[..., :d // 2].abs() + x[..., d // 2:].abs()).amax(-1)
            x = _rotate(x, pos, case["base"])
        else:
            amax = x.abs().amax(-1)
        codes, scales = s[name + "_pages"], s[name + "_scales"]
        need = torch.full_like(scales, -1.0)
        need = need.scatter_reduce(0, pg[:, None].expand_as(amax), amax, "amax")
        want = _scale_of(need.clamp(min=0.0))
        # a page that holds earlier tokens keeps its scale or grows it
        old = torch.zeros_like(scales)
        old = torch.cat([old, old[:1]])
        holds = live & (start % page > 0)
        old[torch.where(holds, first, spare)] = scales[first.clamp(min=0)]
        new = torch.where(need >= 0, torch.maximum(want, old[:-1]), scales)
        ratio = (scales / new)[first.clamp(min=0)][:, :, None, None]
        block = codes[first.clamp(min=0)]
        again = (block.float() * ratio).to(torch.float8_e4m3fn)
        is_old = (torch.arange(page, device=b.device) < (start % page)[:, None])[:, None, :, None]
        raw = codes.view(torch.uint8)
        block = torch.where(is_old & live[:, None, None, None], again.view(torch.uint8),
                            block.view(torch.uint8))
        grown = torch.cat([raw, raw[:1]])
        grown[torch.where(live, first, spare)] = block
        grown[pg, :, slot] = (x / new[pg][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        raw.copy_(grown[:-1])
        scales.copy_(new)
    return {k: s[k] for k in ("k_pages", "v_pages", "k_scales", "v_scales")}


def _attend_plain(s):
    case = s["case"]
    page, d, hq, hkv = case["page"], case["d"], case["hq"], case["hkv"]
    group, most = hq // hkv, max(s["news_host"])
    table = s["page_table"].long().clamp(min=0)
    batch, length = table.shape[0], table.shape[1] * page
    b, i, pos = _tokens(s)
    lens = s["seq_lens"].long()
    at = torch.arange(length, device=b.device)
    held = at < lens[:, None]
    k, v = (((s[n + "_pages"][table].float() * s[n + "_scales"][table][..., None, None])
             .transpose(1, 2).reshape(batch, hkv, length, d)) for n in ("k", "v"))
    v = torch.where(held[:, None, :, None], v, torch.zeros_like(v))
    rows = torch.zeros(batch, most, hq, d, device=b.device)
    rows[b, i] = _rotate(s["q"], pos, case["base"])
    rows = rows.reshape(batch, most, hkv, group, d).permute(0, 2, 3, 1, 4)
    rows = rows.reshape(batch, hkv, group * most, d)
    score = (rows @ k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    where = torch.full((batch, most), -1, dtype=torch.long, device=b.device)
    where[b, i] = pos
    sees = held[:, None, :] & (at <= where[:, :, None])
    if case["window"]:
        sees &= at > where[:, :, None] - case["window"]
    score = score.reshape(batch, hkv, group, most, length)
    score = torch.where(sees[:, None, None], score, torch.full_like(score[:1, :1, :1, :1, :1],
                                                                    -math.inf))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    got = p.reshape(batch, hkv, group * most, length) @ v
    got = got.reshape(batch, hkv, group, most, d)
    got = torch.where(total > 0, got / total, torch.zeros_like(got))
    got = got.permute(0, 3, 1, 2, 4).reshape(batch, most, hq, d)
    s["out"].copy_(got[b, i])
    return s["out"]


def run(s):
    if own:
        pools = s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]
        if s["case"]["kind"] == "append":
            s["cache"].append(s["K_new"], s["V_new"], *pools)
            return {k: s[k] for k in ("k_pages", "v_pages", "k_scales", "v_scales")}
        return s["cache"].attend(s["q"], *pools, out=s["out"])
    return _append_plain(s) if s["case"]["kind"] == "append" else _attend_plain(s)


def _rotate64(x, pos, base):
    half = x.shape[-1] // 2
    power = torch.arange(half, device=x.device, dtype=torch.float64) * (-math.log(base) / half)
    z = torch.complex(x[..., :half], x[..., half:])
    turn = torch.polar(torch.ones(pos.numel(), half, device=x.device, dtype=torch.float64),
                       pos.double()[:, None] * torch.exp(power))
    z = z * turn.reshape([pos.numel()] + [1] * (x.dim() - 2) + [half])
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    s = prepare(case, seed)
    page, d, hq, hkv, window = (case[n] for n in ("page", "d", "hq", "hkv", "window"))
    lens, news, offs = s["seq_lens_host"], s["news_host"], s["offsets_host"]
    dev = s["page_table"].device
    table = s["page_table"].cpu().long()
    if case["kind"] == "append":
        got = {}
        for name in ("k", "v"):
            codes, scales = s[name + "_pages"].double(), s[name + "_scales"].double()
            x = s["K_new" if name == "k" else "V_new"].double()
            for b, (n, m) in enumerate(zip(lens, news)):
                m0 = min(n, m)
                if m0 == 0:
                    continue
                start = n - m0
                rows = x[offs[b] + m - m0:offs[b] + m]
                if name == "k":
                    size = rows[..., :d // 2].abs() + rows[..., d // 2:].abs()
                    rows = _rotate64(rows, torch.arange(start, n, device=dev), case["base"])
                else:
                    size = rows.abs()
                size = size.amax(-1).float()
                for j in range(start // page, (n - 1) // page + 1):
                    lo, hi = max(start, j * page), min(n, (j + 1) * page)
                    pg = int(table[b, j])
                    new = _scale_of(size[lo - start:hi - start].amax(0)).double()
                    if lo > j * page:
                        new = torch.maximum(new, scales[pg])
                        keep = codes[pg, :, :lo - j * page]
                        keep *= (scales[pg] / new)[:, None, None]
                    codes[pg, :, lo - j * page:hi - j * page] = (
                        rows[lo - start:hi - start] / new[:, None]).transpose(0, 1)
                    scales[pg] = new
            got[name + "_pages"], got[name + "_scales"] = codes, scales
        return got
    out = torch.zeros(offs[-1], hq, d, dtype=torch.float64, device=dev)
    group = hq // hkv
    for b, (n, m) in enumerate(zip(lens, news)):
        if n == 0 or m == 0:
            continue
        pages = table[b, :-(-n // page)].to(dev)
        pos = torch.arange(n - m, n, device=dev)
        q = _rotate64(s["q"][offs[b]:offs[b + 1]].double(), pos, case["base"])
        at = torch.arange(n, device=dev)
        hide = at[None] > pos[:, None]
        if window:
            hide |= at[None] <= pos[:, None] - window
        for u in range(hkv):
            k, v = ((s[c + "_pages"][pages, u].double() * s[c + "_scales"][pages, u].double()
                     [:, None, None]).reshape(-1, d)[:n] for c in ("k", "v"))
            for h in range(u * group, (u + 1) * group):
                w = (q[:, h] @ k.T) / math.sqrt(d)
                w.masked_fill_(hide, -math.inf)
                w = torch.softmax(w, -1)
                if m > n:
                    w = torch.nan_to_num(w)
                out[offs[b]:offs[b + 1], h] = w @ v
    return out
