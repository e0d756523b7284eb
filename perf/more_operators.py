"""The operators that chunks, capped and biased scores and moved sequences need beside the 2-bit KV cache, as cases
that can be timed and compared.

Five operators, each in a plain form (elementary torch operations in 32 bits) and, where `own` is true, as the
library's call.  The score rule of the first three: x = scale q . k, capped to cap tanh(x / cap) where there is a cap,
less slope[head] |distance in tokens| where there are slopes.

  chunk    attention within a new chunk: packed documents, each token over the keys of its own document up to itself
           (or up to the document's prefix, which every token sees), merged with the rows that the same queries got
           over what precedes the chunk
  history  the chunk's queries over every token already in the 2-bit cache, under the rule
  decode   single-token attention over the 2-bit cache, under the rule
  fork     the first tokens of sequences copied to other slots of the cache; where a copy ends inside a packed group,
           its tokens there continue as bf16 window rows
  keep     sequences compacted to listed groups and their window, into another slot or (after a fork) in place

The cache's bytes (include/oscar.h: group blocks of 128 tokens) are made here with torch, so both forms see the same
packed groups.
"""
import math

import torch

own = False

D = 128          # head dimension
G = 128          # tokens per group


def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _gen(seed, salt=0):
    g = torch.Generator(device=_device())
    g.manual_seed(1000003 * int(seed) + salt)
    return g


def _dtype(case):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[case["type"]]


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # 8 sequences verify 5 drafted tokens each, their rows over the cache merged in: launch latency
        dict(name="chunk_verify", op="chunk", docs=8, length=5, ragged=False, hkv=8, gqa=4, cap=0.0, bias=False,
             prefix=False, prior=True, fused=False),
        # a packed batch of short prompts of a model with capped scores
        dict(name="chunk_docs_capped", op="chunk", docs=24, length=1531, ragged=True, hkv=8, gqa=4, cap=50.0,
             bias=False, prefix=False, prior=False, fused=True),
        # prompts whose first part is read in both directions, with distance biases, a KV head for each query head
        dict(name="chunk_prefix_bias", op="chunk", docs=3, length=4099, ragged=True, hkv=16, gqa=1, cap=0.0, bias=True,
             prefix=True, prior=False, fused=False),
        # a prefill chunk of 8K tokens straight out of a fused projection, its history merged in
        dict(name="chunk_8k", op="chunk", docs=1, length=8192, ragged=False, hkv=8, gqa=4, cap=0.0, bias=False,
             prefix=False, prior=True, fused=True),
        # 512 new queries over a history of 32K tokens, capped
        dict(name="history_512x32k_capped", op="history", n=512, hkv=8, gqa=4, length=32768, meta=32, cap=30.0,
             bias=False),
        # the last odd piece of a prompt, 5 query heads a KV head, distance biases, 16-bit metadata, a window of 15
        dict(name="history_odd_bias", op="history", n=77, hkv=4, gqa=5, length=9999, meta=16, cap=0.0, bias=True),
        # a decode step at 128K, capped
        dict(name="decode_128k_capped", op="decode", b=1, hkv=8, gqa=4, length=131072 - 51, ragged=False, meta=32,
             type="bf16", cap=30.0, bias=False),
        # a ragged batch, 8 query heads a KV head, both rules, 16-bit metadata, float32 outputs
        dict(name="decode_ragged_gqa8", op="decode", b=7, hkv=4, gqa=8, length=20011, ragged=True, meta=16, type="f32",
             cap=20.0, bias=True),
        # four continuations of one 128K prompt
        dict(name="fork_128k_x4", op="fork", b=4, shared=True, hkv=8, length=131072 - 51, ragged=False, meta=32,
             cut=False),
        # prefixes of cached prompts taken over by new requests, each ending inside a group
        dict(name="fork_prefixes", op="fork", b=6, shared=False, hkv=4, length=9001, ragged=True, meta=16, cut=True),
        # a 128K sequence pruned to its first and its latest groups
        dict(name="keep_128k_recent", op="keep", b=1, hkv=8, length=131072 - 51, ragged=False, meta=32, keep=512,
             scattered=False, inplace=False),
        # a batch forked and pruned in place to scattered groups
        dict(name="keep_scattered_inplace", op="keep", b=16, hkv=8, length=16384 + 77, ragged=True, meta=32, keep=64,
             scattered=True, inplace=True),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "history", "decode", "fork", "keep"])
    hkv = rng.choice([1, 2, 4, 8])
    gqa = rng.choice([1, 2, 3, 4, 5, 8])
    meta = rng.choice([32, 32, 16])
    ragged = rng.random() < 0.5
    rule = dict(cap=rng.choice([0.0, 0.0, 20.0, 50.0]), bias=rng.random() < 0.4)
    if op == "chunk":
        # at most the score pairs and the rows of chunk_8k
        docs = _log(rng, 1, 32)
        most = int(min(8192.0 / docs, 8192.0 * math.sqrt(32.0 / (docs * hkv * gqa))))
        return dict(op=op, docs=docs, length=_log(rng, 1, most), ragged=ragged, hkv=hkv, gqa=gqa,
                    prefix=rng.random() < 0.3, prior=rng.random() < 0.5, fused=rng.random() < 0.5, **rule)
    if op == "history":
        n = _log(rng, 1, 512)
        most = 512 * 32 * 32768 // (n * hkv * gqa)
        return dict(op=op, n=n, hkv=hkv, gqa=gqa, length=_log(rng, 60, min(32768, most)), meta=meta, **rule)
    if op == "decode":
        b = _log(rng, 1, 32)
        return dict(op=op, b=b, hkv=hkv, gqa=gqa, length=_log(rng, 60, min(131072, 131072 * 8 // (b * hkv))),
                    ragged=ragged, meta=meta, type=rng.choice(["bf16", "bf16", "f32"]), **rule)
    b = _log(rng, 1, 16)
    length = _log(rng, 60, min(131072, (20 if op == "fork" else 10) * 131072 // (b * hkv)))
    if op == "fork":
        return dict(op=op, b=b, shared=rng.random() < 0.4, hkv=hkv, length=length, ragged=ragged, meta=meta,
                    cut=rng.random() < 0.5)
    length = max(length, 300)
    return dict(op=op, b=b, hkv=hkv, length=length, ragged=ragged, meta=meta, keep=_log(rng, 1, length // G),
                scattered=rng.random() < 0.5, inplace=rng.random() < 0.5)


def _lengths(case):
    """Tokens of each sequence: all `length`, or spread below it (the first one whole), odd ones among them."""
    b = case.get("b", case.get("docs", 1))
    if not case.get("ragged"):
        return [case["length"]] * b
    n = case["length"]
    return [max(1, n - (i * n) // b - 13 * i) for i in range(b)]


def _prefixes(case, lens):
    """Tokens that a document's every token sees: a third of the first, less of the others, none of the last."""
    return [(n // (3 + i) if i + 1 < len(lens) or i == 0 else 0) for i, n in enumerate(lens)]


def _pairs(case):
    """Visible (token, key) pairs of a chunk."""
    lens = _lengths(case)
    pre = _prefixes(case, lens) if case["prefix"] else [0] * len(lens)
    return sum(n * (n + 1) // 2 + p * (p - 1) // 2 for n, p in zip(lens, pre))


def _forks(case):
    """(source slot, tokens taken) of each fork: `b` forks of one sequence, or one of each."""
    lens = [case["length"]] if case["shared"] else _lengths(case)
    out = []
    for i in range(case["b"]):
        src = 0 if case["shared"] else i
        n = lens[src]
        out.append((src, max(1, n - n // 5 - 37 - 11 * i) if case["cut"] else n))
    return lens, out


def _kept(case):
    """Groups that each sequence keeps, ascending: the first two and the latest, or every so many."""
    out = []
    for i, n in enumerate(_lengths(case)):
        ng = n // G
        m = min(case["keep"], ng)
        if case["scattered"]:
            out.append([(t * ng) // m for t in range(m)])
        else:
            first = min(2, m)
            out.append(list(range(first)) + list(range(ng - (m - first), ng)))
    return out


def work(case):
    op, hkv = case["op"], case["hkv"]
    if op == "chunk":
        rows, hq = sum(_lengths(case)), hkv * case["gqa"]
        bytes_ = rows * (hq * (D * 4 + 4) + 2 * hkv * D * 2) + (rows * hq * (D * 2 + 4) if case["prior"] else 0)
        return {"bytes": bytes_, "flops": 4 * D * hq * _pairs(case)}
    block = 13824 if case["meta"] == 32 else 11008
    if op == "history":
        hq, n = hkv * case["gqa"], case["length"]
        return {"bytes": hkv * (n // G * block + n % G * 4 * D) + case["n"] * hq * (D * 4 + 4),
                "flops": 4 * D * hq * case["n"] * n}
    if op == "decode":
        lens, hq = _lengths(case), hkv * case["gqa"]
        out = 2 if case["type"] == "bf16" else 4
        return {"bytes": sum(hkv * (n // G * block + n % G * 4 * D) for n in lens) + case["b"] * hq * D * (2 + out),
                "flops": 4 * D * hq * sum(lens)}
    if op == "fork":
        lens, forks = _forks(case)
        size = lambda n: hkv * (n // G * block + n % G * 4 * D + 8)  # noqa: E731
        read = size(max(n for _, n in forks)) if case["shared"] else sum(size(n) for _, n in forks)
        return {"bytes": read + sum(size(n) for _, n in forks), "flops": 0}
    lens, kept = _lengths(case), _kept(case)
    total = 0
    for n, k in zip(lens, kept):
        window = n % G * 4 * D + 8
        if case["inplace"]:     # the fork, then the groups that change their place
            total += 2 * hkv * (n // G * block + window)
            total += 2 * hkv * block * sum(1 for i, g in enumerate(k) if g != i)
        else:
            total += 2 * hkv * (len(k) * block + window)
    return {"bytes": total, "flops": 0}


# ------------------------------------------------ packed groups, as stored

def _hadamard(dtype, device):
    """Unnormalised Sylvester matrix, entry (-1)^popcount(i & j)."""
    h = torch.ones((1, 1), dtype=dtype, device=device)
    for _ in range(7):
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _token_rows(device):
    """Row of each token in the float32 value metadata."""
    t = torch.arange(G, device=device)
    return t ^ ((t >> 3) & 1)


def _pack(codes, value_order):
    """uint8 codes [N, 128 rows, 128 columns] -> the 4,096 bytes of each matrix."""
    n = codes.shape[0]
    c = codes.view(n, 8, 2, 8, 2, 2, 2, 2, 4, 2)         # mt r g | j kh kl hf tig e
    if value_order:
        c = c.permute(0, 1, 4, 3, 8, 2, 9, 5, 6, 7)      # mt j g tig r e kh | kl hf
    else:
        c = c.permute(0, 1, 3, 8, 4, 2, 9, 5, 6, 7)      # mt g tig j r e kh | kl hf
    b = c[..., 0, 0] | (c[..., 0, 1] << 2) | (c[..., 1, 0] << 4) | (c[..., 1, 1] << 6)
    return b.reshape(n, 4096)


def _quantise(x, dim, meta):
    """Asymmetric 2-bit codes with stored scale and zero along `dim` of x."""
    lo, hi = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    s, z = (hi - lo) / 3.0, lo
    if meta == 16:
        s, z = s.half().float(), z.half().float()
    q = torch.where(s > 0, torch.round((x - z) / s), torch.zeros_like(x)).clamp_(0, 3)
    return q.to(torch.uint8), s, z


def _groups(n, heads, first, meta, gen):
    """n random groups as stored bytes, [n, block]; group i belongs to row heads[i], first[i]: a sequence's first group."""
    dev = _device()
    block = 13824 if meta == 32 else 11008
    raw = torch.empty((n, block), dtype=torch.uint8, device=dev)
    h = _hadamard(torch.float32, dev) / math.sqrt(D)
    rows = int(heads.max()) + 1 if n else 0
    loud = torch.ones((rows, D), device=dev)
    loud.scatter_(1, torch.randint(0, D, (rows, 4), device=dev, generator=gen), 15.0)
    vloud = torch.ones((rows, D), device=dev)
    vloud.scatter_(1, torch.randint(0, D, (rows, 2), device=dev, generator=gen), 5.0)
    for a in range(0, n, 8192):
        m = min(8192, n - a)
        row = heads[a:a + m]
        k = torch.randn((m, G, D), device=dev, generator=gen)
        k += 0.6 * torch.randn((m, 1, D), device=dev, generator=gen)          # what the group is about
        k *= loud[row][:, None] * torch.exp(0.5 * torch.randn((m, G, 1), device=dev, generator=gen))
        k[:, 0] *= torch.where(first[a:a + m], 0.05, 1.0)[:, None]            # the sink
        k = k.bfloat16().float()
        norm = k.norm(dim=2, keepdim=True)
        unit = (k / norm) @ h
        if meta == 16:
            norm = norm.half().float()
        kc, ks, kz = _quantise(unit, 1, meta)
        v = (torch.randn((m, G, D), device=dev, generator=gen) * vloud[row][:, None]).bfloat16().float()
        vc, vs, vz = _quantise(v.view(m, G, 4, 32), 3, meta)
        t = torch.float16 if meta == 16 else torch.float32
        order = _token_rows(dev) if meta == 32 else torch.arange(G, device=dev)
        store = lambda x: x.reshape(m, -1).to(t).contiguous().view(torch.uint8)  # noqa: E731
        raw[a:a + m] = torch.cat([_pack(kc, False), store(ks), store(kz), store(norm),
                                  _pack(vc.view(m, G, D).transpose(1, 2).contiguous(), True),
                                  store(vs.view(m, G, 4)[:, order]), store(vz.view(m, G, 4)[:, order])], 1)
    return raw


def _cache(case, lens, seed):
    """A batch's packed groups [b, hkv, groups, block], windows [b, hkv, 2, 128, 128] and value maxima [b, 2, hkv]."""
    dev, hkv = _device(), case["hkv"]
    b, ng = len(lens), max(lens) // G
    gen = _gen(seed, 1)
    heads = torch.arange(b * hkv, device=dev).repeat_interleave(ng)
    first = torch.arange(ng, device=dev).repeat(b * hkv) == 0
    raw = _groups(b * hkv * ng, heads, first, case["meta"], gen).view(b, hkv, ng, 13824 if case["meta"] == 32 else 11008)
    window = torch.randn((b, hkv, 2, G, D), device=dev, generator=gen).bfloat16()
    t, start = (torch.float32, 9728) if case["meta"] == 32 else (torch.float16, 8960)
    meta = raw[..., start:].contiguous().view(t).float().view(b, hkv, ng, 2, 4 * G)
    live = torch.arange(ng, device=dev) < (torch.tensor(lens, device=dev) // G)[:, None]
    top = (meta.abs().amax(-1) * live[:, None, :, None]).amax(2) if ng else torch.zeros((b, hkv, 2), device=dev)
    return raw, window, top.transpose(1, 2).contiguous()


def _codes(raw, value_order):
    """The 4,096 bytes of each code matrix, [..., 4096] -> codes [..., 128 tokens, 128 channels] (float32)."""
    lead = raw.shape[:-1]
    c = (raw.unsqueeze(-1) >> torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=raw.device)) & 3
    if value_order:
        c = c.reshape(-1, 8, 2, 8, 4, 2, 2, 2, 2, 2).permute(0, 2, 7, 8, 9, 4, 6, 1, 5, 3)   # token first
    else:
        c = c.reshape(-1, 8, 8, 4, 2, 2, 2, 2, 2, 2).permute(0, 1, 5, 2, 4, 7, 8, 9, 3, 6)
    return c.reshape(lead + (G, D)).float()


def _split(raw, meta):
    """Stored blocks [..., block] -> rotated keys [..., 128, 128] and values [..., 128, 128], float32."""
    t, at = (torch.float32, (4096, 4608, 5120, 5632, 9728, 11776, 13824)) if meta == 32 else \
        (torch.float16, (4096, 4352, 4608, 4864, 8960, 9984, 11008))
    part = lambda i: raw[..., at[i]:at[i + 1]].contiguous().view(t).float()  # noqa: E731
    k = (_codes(raw[..., :4096], False) * part(0).unsqueeze(-2) + part(1).unsqueeze(-2)) * part(2).unsqueeze(-1)
    order = _token_rows(raw.device) if meta == 32 else torch.arange(G, device=raw.device)
    vs = part(4).unflatten(-1, (G, 4))[..., order, :].repeat_interleave(32, -1)
    vz = part(5).unflatten(-1, (G, 4))[..., order, :].repeat_interleave(32, -1)
    v = _codes(raw[..., at[3]:at[4]], True) * vs + vz
    return k, v


# ------------------------------------------------------- inputs of each case

def _slopes(case):
    """Distance slopes of the query heads: a geometric series down to 2^-8."""
    hq = case["hkv"] * case["gqa"]
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], dtype=torch.float32, device=_device())


def _rule(case):
    return dict(cap=case["cap"], slopes=_slopes(case) if case["bias"] else None)


def _own_cache(case, lens, raw, window, top, slots, longest):
    from int2_kv_cache_oscar_gb300 import oscar as O
    cache = O.OscarCache(slots, case["hkv"], longest, meta_bits=case["meta"])
    for i, n in enumerate(lens):
        cache.import_sequence(i, n, raw[i, :, :n // G].contiguous(), window[i], top[i])
    return O, cache


def _chunk_inputs(case, seed):
    """q, k, v of the packed tokens (views of one fused projection where the case says so), and the rows to merge."""
    dev, gen, hkv, hq = _device(), _gen(seed, 2), case["hkv"], case["hkv"] * case["gqa"]
    n = sum(_lengths(case))
    x = torch.randn((n, hq + 2 * hkv, D), device=dev, generator=gen)
    x[:, hq:hq + hkv] += 0.5 * torch.randn((1, hkv, D), device=dev, generator=gen)      # keys share a direction
    loud = torch.ones((hkv, D), device=dev)
    loud.scatter_(1, torch.randint(0, D, (hkv, 4), device=dev, generator=gen), 6.0)     # and have loud channels
    x[:, hq:hq + hkv] *= loud
    x = x.bfloat16()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if not case["fused"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    prior = None
    if case["prior"]:
        po = torch.randn((n, hq, D), device=dev, generator=gen).mul_(0.2).bfloat16()
        pl = torch.randn((n, hq), device=dev, generator=gen) + math.log(1.0 + _lengths(case)[0])
        if len(_lengths(case)) > 1:                                                     # a sequence without a history
            pl[:_lengths(case)[0]] = -math.inf
        prior = (po, pl)
    return q, k, v, prior


def _queries(case, seed, n):
    return torch.randn((n, case["hkv"] * case["gqa"], D), device=_device(), generator=_gen(seed, 3)).bfloat16()


def _cumulative(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _views(cache, slot, length):
    """A slot's group blocks, window rows and maxima within the arena: the state's own buffers."""
    from int2_kv_cache_oscar_gb300 import oscar as O
    hkv, block, arena = cache.num_kv_heads, cache.block_bytes, cache.arena
    groups = (cache.max_seq_len + G - 1) // G
    at = O.oscar_cache_block_offset(cache.handle, slot, 0, 0)
    blocks = arena.as_strided((hkv, length // G, block), (groups * block, block, 1), at)
    at = O.oscar_cache_window_offset(cache.handle, slot, 0)
    window = arena[at:at + hkv * 65536].view(torch.bfloat16).view(hkv, 2, G, D)[:, :, :length % G]
    top = arena.view(torch.float32).as_strided((2, hkv), (cache.max_batch * hkv, 1), 64 + slot * hkv)
    return blocks, window, top


def prepare(case, seed):
    op, st = case["op"], dict(case=case)
    if op == "chunk":
        q, k, v, prior = _chunk_inputs(case, seed)
        lens = _lengths(case)
        st.update(q=q, k=k, v=v, prior=prior, cu=_cumulative(lens), prefix=_prefixes(case, lens) if case["prefix"] else None,
                  rule=_rule(case))
        if own:
            from int2_kv_cache_oscar_gb300 import oscar as O
            st["O"] = O
            st["out"] = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            st["lse"] = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
        return st
    if op in ("history", "decode"):
        lens = [case["length"]] if op == "history" else _lengths(case)
        raw, window, top = _cache(case, lens, seed)
        n = case["n"] if op == "history" else len(lens)
        st.update(q=_queries(case, seed, n), lens=lens, rule=_rule(case))
        if own:
            O, st["cache"] = _own_cache(case, lens, raw, window, top, len(lens), max(lens))
            hq = st["q"].shape[1]
            if op == "history":
                st["out"], st["lse"] = torch.empty_like(st["q"]), torch.empty((n, hq), device=raw.device)
                size = O.oscar_prefill_workspace_bytes(st["cache"].handle, 0, n, hq)
                st["workspace"] = torch.empty(size, dtype=torch.uint8, device=raw.device) if size else None
            else:
                st["out"] = torch.empty(st["q"].shape, dtype=_dtype(case), device=raw.device)
                st["workspace"] = st["cache"].workspace(n, hq)
        else:
            st["raw"], st["window"] = raw, window
        return st
    lens = _forks(case)[0] if op == "fork" else _lengths(case)
    raw, window, top = _cache(case, lens, seed)
    b = case["b"]
    st.update(lens=lens)
    if op == "fork":
        st["src"], st["take"] = [s for s, _ in _forks(case)[1]], [n for _, n in _forks(case)[1]]
    else:
        st["src"], st["kept"] = list(range(b)), _kept(case)
        st["take"] = [len(g) * G + n % G for g, n in zip(st["kept"], lens)]
    if own:
        st["dst"] = [len(lens) + i for i in range(b)]
        _, st["cache"] = _own_cache(case, lens, raw, window, top, len(lens) + b, max(lens))
        st["made"] = [_views(st["cache"], s, n) for s, n in zip(st["dst"], st["take"])]
    else:
        st["raw"], st["window"], st["top"] = raw, window, top
        if op == "keep":
            st["rows"] = [torch.tensor(g, dtype=torch.long, device=raw.device) for g in st["kept"]]
    return st


# --------------------------------------------------------------- one pass

def run(state):
    return {"chunk": _run_chunk, "history": _run_history, "decode": _run_decode, "fork": _run_fork,
            "keep": _run_keep}[state["case"]["op"]](state)


def _score(x, q_pos, k_pos, rule, hkv):
    """The score rule on x [hkv, gqa, queries, keys] (scaled products), positions [queries] and [keys]."""
    if rule["cap"]:
        x = rule["cap"] * torch.tanh(x / rule["cap"])
    if rule["slopes"] is not None:
        far = (q_pos[:, None] - k_pos[None, :]).abs().to(x.dtype)
        x = x - rule["slopes"].to(x.dtype).view(hkv, -1, 1, 1) * far
    return x


def _run_chunk(st):
    case, prior = st["case"], st["prior"]
    if own:
        po, pl = prior if prior is not None else (None, None)
        st["O"].oscar_chunk_attention(st["cu"], st["q"], st["k"], st["v"], st["out"], st["lse"], prefix=st["prefix"],
                                      cap=st["rule"]["cap"], slopes=st["rule"]["slopes"], prior_out=po, prior_lse=pl)
        return {"out": st["out"], "lse": st["lse"]}
    hkv = case["hkv"]
    out, lse = torch.empty(st["q"].shape, dtype=torch.float32, device=st["q"].device), \
        torch.empty(st["q"].shape[:2], dtype=torch.float32, device=st["q"].device)
    for d in range(len(st["cu"]) - 1):
        a, e = st["cu"][d], st["cu"][d + 1]
        q = st["q"][a:e].float().unflatten(1, (hkv, -1)).permute(1, 2, 0, 3)           # [hkv, gqa, n, 128]
        k, v = (st[x][a:e].float().transpose(0, 1)[:, None] for x in ("k", "v"))       # [hkv, 1, n, 128]
        at = torch.arange(e - a, device=q.device)
        x = _score(q @ k.transpose(-1, -2) * (1.0 / math.sqrt(D)), at, at, st["rule"], hkv)
        end = at + 1 if st["prefix"] is None else (at + 1).clamp_min(st["prefix"][d])
        x = x.masked_fill(at[None, :] >= end[:, None], -math.inf)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - m)
        l = p.sum(-1, keepdim=True)
        out[a:e] = (p @ v / l).permute(2, 0, 1, 3).flatten(1, 2)
        lse[a:e] = (m + torch.log(l)).squeeze(-1).permute(2, 0, 1).flatten(1, 2)
    if prior is not None:
        both = torch.maximum(lse, prior[1])
        w1, w0 = torch.exp(lse - both), torch.exp(prior[1] - both)
        out = (out * w1[..., None] + prior[0].float() * w0[..., None]) / (w1 + w0)[..., None]
        lse = both + torch.log(w1 + w0)
    return {"out": out.to(st["q"].dtype), "lse": lse}


def _rows_of(raw, window, length, meta):
    """Rotated keys and values of one sequence's groups, and its window's rows: [hkv, tokens, 128] each."""
    k, v = _split(raw[:, :length // G], meta)
    return k.flatten(1, 2), v.flatten(1, 2), window[:, 0, :length % G].float(), window[:, 1, :length % G].float()


def _attend(q, raw, window, length, q_pos, rule, meta):
    """q [hkv, gqa, n, 128] over a sequence: outputs [hkv, gqa, n, 128] and log-sum-exp."""
    hkv = q.shape[0]
    k, v, wk, wv = _rows_of(raw, window, length, meta)
    turned = q @ (_hadamard(torch.float32, q.device) / math.sqrt(D))
    x = torch.cat([turned @ k[:, None].transpose(-1, -2), q @ wk[:, None].transpose(-1, -2)], -1) * (1.0 / math.sqrt(D))
    x = _score(x, q_pos, torch.arange(length, device=q.device), rule, hkv)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    return p @ torch.cat([v, wv], 1)[:, None] / l, (m + torch.log(l)).squeeze(-1)


def _run_history(st):
    case = st["case"]
    if own:
        st["cache"].scored_prefill(0, st["q"], st["q"].shape[1], st["out"], st["lse"], st["workspace"], **st["rule"])
        return {"out": st["out"], "lse": st["lse"]}
    n, length = case["n"], case["length"]
    q = st["q"].float().unflatten(1, (case["hkv"], -1)).permute(1, 2, 0, 3)
    at = length + torch.arange(n, device=q.device)
    o, lse = _attend(q, st["raw"][0], st["window"][0], length, at, st["rule"], case["meta"])
    return {"out": o.permute(2, 0, 1, 3).flatten(1, 2).to(st["q"].dtype), "lse": lse.permute(2, 0, 1).flatten(1, 2)}


def _run_decode(st):
    case = st["case"]
    if own:
        st["cache"].scored_decode(list(range(len(st["lens"]))), st["q"], st["q"].shape[1], st["out"], st["workspace"],
                                  **st["rule"])
        return st["out"]
    q = st["q"].float().unflatten(1, (case["hkv"], -1))
    rows = []
    for i, n in enumerate(st["lens"]):
        at = torch.tensor([n - 1], device=q.device)
        rows.append(_attend(q[i][:, :, None], st["raw"][i], st["window"][i], n, at, st["rule"], case["meta"])[0][:, :, 0])
    return torch.stack(rows).flatten(1, 2).to(_dtype(case))


def _run_fork(st):
    case = st["case"]
    if own:
        st["cache"].fork(st["src"], st["dst"], st["take"])
        return st["made"]
    out = []
    for s, n in zip(st["src"], st["take"]):
        have, ng = st["lens"][s], n // G
        blocks = st["raw"][s, :, :ng].clone()
        if n % G and have // G > ng:          # ends inside a packed group: its tokens in bf16
            k, v = _split(st["raw"][s, :, ng], case["meta"])
            k = k @ (_hadamard(torch.float32, k.device) / math.sqrt(D))
            window = torch.stack([k, v], 1)[:, :, :n % G].bfloat16()
        else:
            window = st["window"][s][:, :, :n % G].clone()
        out.append([blocks, window, st["top"][s].clone()])
    return out


def _run_keep(st):
    case = st["case"]
    if own:
        if case["inplace"]:
            st["cache"].fork(st["src"], st["dst"])
            st["cache"].keep_groups(st["dst"], st["kept"])
        else:
            st["cache"].keep_groups(st["src"], st["kept"], st["dst"])
        return st["made"]
    raw = st["raw"].clone() if case["inplace"] else st["raw"]
    return [[raw[i].index_select(1, rows), st["window"][i][:, :, :n % G].clone(), st["top"][i].clone()]
            for i, (rows, n) in enumerate(zip(st["rows"], st["lens"]))]


# ------------------------------------------- the definitions, in 64 bits

_tables = {}


def _bit_table(value_order, device):
    """Byte and bit of every code: [128 tokens, 128 channels] each, from the layout's description."""
    if (value_order, str(device)) not in _tables:
        row, col = torch.meshgrid(torch.arange(128), torch.arange(128), indexing="ij")
        if value_order:
            row, col = col, row                     # the stored matrix is [channel][token]
        mt, g, r = row // 16, row % 8, (row // 8) % 2
        j, kk, hf, tig, e = col // 64, (col // 16) % 4, (col // 8) % 2, (col // 2) % 4, col % 2
        lane = 4 * g + tig
        word = ((mt * 2 + j) * 32 + lane) * 2 + r if value_order else (mt * 32 + lane) * 4 + 2 * j + r
        bit = 16 * e + 4 * kk + 2 * hf
        _tables[value_order, str(device)] = ((word * 4 + bit // 8).reshape(-1).to(device), (bit % 8).reshape(-1).to(device))
    return _tables[value_order, str(device)]


def _exact_blocks(raw, meta):
    """Stored blocks [n, block] -> rotated keys and values [n, 128, 128] in 64 bits."""
    n, wide = raw.shape[0], meta == 32
    sections, at = [], 0
    for name, size in (("kc", 4096), ("ks", 128), ("kz", 128), ("kn", 128), ("vc", 4096), ("vs", 512), ("vz", 512)):
        size = size if name in ("kc", "vc") else size * (4 if wide else 2)
        piece = raw[:, at:at + size].contiguous()
        sections.append(piece if name in ("kc", "vc") else piece.view(torch.float32 if wide else torch.float16).double())
        at += size
    kc, ks, kz, kn, vc, vs, vz = sections
    byte, bit = _bit_table(False, raw.device)
    k = ((kc[:, byte].long() >> bit) & 3).double().view(n, G, D)
    k = kn[:, :, None] * (k * ks[:, None, :] + kz[:, None, :])
    byte, bit = _bit_table(True, raw.device)
    v = ((vc[:, byte].long() >> bit) & 3).double().view(n, G, 4, 32)
    token = torch.arange(G, device=raw.device)
    where = torch.where((token // 8) % 2 == 1, token - 2 * (token % 2) + 1, token) if wide else token
    vs, vz = vs.view(n, G, 4)[:, where], vz.view(n, G, 4)[:, where]
    return k, (v * vs[..., None] + vz[..., None]).view(n, G, D)


def exact(case, seed):
    return {"chunk": _exact_chunk, "history": _exact_history, "decode": _exact_decode, "fork": _exact_moved,
            "keep": _exact_moved}[case["op"]](case, seed)


def _weigh(s, dist, case, h, hide=None):
    """Softmax weights and log-sum-exp of one head's scaled products s [queries, keys], from the rule's definition."""
    if case["cap"]:
        s = torch.tanh(s / case["cap"]) * case["cap"]
    if case["bias"]:
        s = s - float(_slopes(case)[h]) * dist
    if hide is not None:
        s = torch.where(hide, torch.full_like(s, -math.inf), s)
    return torch.softmax(s, -1), torch.logsumexp(s, -1)


def _exact_chunk(case, seed):
    q, k, v, prior = _chunk_inputs(case, seed)
    lens = _lengths(case)
    cu, pre = _cumulative(lens), _prefixes(case, lens)
    out, lse = q.double(), torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
    for d, n in enumerate(lens):
        a = cu[d]
        i = torch.arange(n, device=q.device)
        hide = i[None, :] > i[:, None]
        if case["prefix"]:
            hide &= (i >= pre[d])[None, :]
        dist = (i[:, None] - i[None, :]).abs().double() if case["bias"] else None
        for h in range(q.shape[1]):
            j = h // case["gqa"]
            s = q[a:a + n, h].double() @ k[a:a + n, j].double().T / math.sqrt(D)
            p, z = _weigh(s, dist, case, h, hide)
            out[a:a + n, h], lse[a:a + n, h] = p @ v[a:a + n, j].double(), z
    if prior is not None:
        total = torch.logaddexp(lse, prior[1].double())
        out = torch.exp(lse - total)[..., None] * out + torch.exp(prior[1].double() - total)[..., None] * prior[0].double()
        lse = total
    return {"out": out, "lse": lse}


def _exact_rows(raw, window, length, meta, j):
    """Keys (in the basis in which they were appended) and values of a sequence's KV head j, [tokens, 128]."""
    h = _hadamard(torch.float64, raw.device)
    ks, vs = [], []
    for c in range(0, length // G, 256):
        k, v = _exact_blocks(raw[j, c:min(c + 256, length // G)], meta)
        ks.append(k.view(-1, D) @ h / math.sqrt(D))
        vs.append(v.view(-1, D))
    ks.append(window[j, 0, :length % G].double())
    vs.append(window[j, 1, :length % G].double())
    return torch.cat(ks), torch.cat(vs)


def _exact_history(case, seed):
    n, length, gqa = case["n"], case["length"], case["gqa"]
    raw, window, _ = _cache(case, [length], seed)
    q = _queries(case, seed, n).double()
    out, lse = q.clone(), torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
    dist = (length + torch.arange(n, device=q.device))[:, None] - torch.arange(length, device=q.device)
    for h in range(q.shape[1]):
        if h % gqa == 0:
            k, v = _exact_rows(raw[0], window[0], length, case["meta"], h // gqa)
        p, lse[:, h] = _weigh(q[:, h] @ k.T / math.sqrt(D), dist.double(), case, h)
        out[:, h] = p @ v
    return {"out": out, "lse": lse}


def _exact_decode(case, seed):
    lens, gqa = _lengths(case), case["gqa"]
    raw, window, _ = _cache(case, lens, seed)
    q = _queries(case, seed, len(lens)).double()
    out = q.clone()
    for i, n in enumerate(lens):
        dist = (n - 1 - torch.arange(n, device=q.device)).double()[None]
        for h in range(q.shape[1]):
            if h % gqa == 0:
                k, v = _exact_rows(raw[i], window[i], n, case["meta"], h // gqa)
            p, _ = _weigh(q[i, h][None] @ k.T / math.sqrt(D), dist, case, h)
            out[i, h] = (p @ v)[0]
    return out


def _exact_moved(case, seed):
    """Bytes of the blocks and values of the window rows that each destination holds."""
    lens, forks = _forks(case) if case["op"] == "fork" else (_lengths(case), None)
    raw, window, top = _cache(case, lens, seed)
    out = []
    for i in range(case["b"]):
        s, n = forks[i] if forks else (i, lens[i])
        groups = list(range(n // G)) if forks else _kept(case)[i]
        blocks = torch.stack([raw[s, :, g] for g in groups], 1) if groups else raw[s, :, :0]
        rows = window[s][:, :, :n % G].double()
        if n % G and lens[s] // G > n // G:
            h = _hadamard(torch.float64, raw.device)
            k, v = _exact_blocks(raw[s, :, n // G], case["meta"])
            rows = torch.stack([k @ h / math.sqrt(D), v], 1)[:, :, :n % G]
        out.append([blocks, rows, top[s].double()])
    return out
