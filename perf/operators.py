"""The operators around the 2-bit KV cache, as cases that can be timed and compared.

Four operators, each in a plain form (elementary torch operations in 32 bits)
and, where `own` is true, as the library's call:

  rotary   rotary positions of the queries and keys that the cache takes
           (half and interleaved layouts, part of the head, scaled for long
           contexts, and the transpose, which is its gradient)
  read     tokens of the cache read back: 2-bit groups dequantised (keys
           rotated back to their own basis), the bf16 window as it is
  select   the groups that are worth attending for each new query: a cheap
           score from an 8-bit summary of each group's key range, then the
           largest scores of each KV head, lowest group first on a tie
  sparse   single-token attention over the listed groups and the window

The cache's bytes (include/oscar.h: group blocks of 128 tokens) are made here
with torch, so both forms see the same packed groups.
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
        # one decode step's rotation for the 32 query / 8 KV head layer: launch latency
        dict(name="rotary_step", op="rotary", n=1, hq=32, hkv=8, type="bf16", dim=128, interleaved=False,
             scaling="banded", factor=8.0, base=500000.0, first=131000, fused=True, transpose=False),
        # a prefill chunk at far positions, straight out of a fused projection
        dict(name="rotary_chunk", op="rotary", n=8192, hq=32, hkv=8, type="bf16", dim=128, interleaved=False,
             scaling="banded", factor=8.0, base=500000.0, first=122880, fused=True, transpose=False),
        # the gradient of a partial, interleaved rotation in float32, an odd number of tokens
        dict(name="rotary_grad_partial", op="rotary", n=2053, hq=16, hkv=4, type="f32", dim=64, interleaved=True,
             scaling="yarn", factor=4.0, base=10000.0, first=30000, fused=False, transpose=True),
        # a short sequence of one KV head read back whole: 8 groups and a 37-token window
        dict(name="read_short", op="read", b=1, hkv=1, length=1061, ragged=False, meta=32, type="bf16", part=False),
        # the 128K context of the 8-head layer read back, as to hand it to dense attention
        dict(name="read_128k", op="read", b=1, hkv=8, length=131072, ragged=False, meta=32, type="bf16", part=False),
        # parts of a ragged batch in float32 from the 16-bit metadata layout, starting and ending inside groups
        dict(name="read_ragged_f32", op="read", b=5, hkv=4, length=30011, ragged=True, meta=16, type="f32", part=True),
        # a decode step at 8K: 64 groups a head, a quarter kept
        dict(name="select_8k", op="select", b=1, hkv=8, gqa=4, length=8192, ragged=False, meta=32, keep=16, update=False),
        # a batch of 32 at 32K: 256 rows, a quarter kept
        dict(name="select_b32_32k", op="select", b=32, hkv=8, gqa=4, length=32768, ragged=False, meta=32, keep=64,
             update=False),
        # the first step after the prefill of a ragged batch: every group is summarised first
        dict(name="select_after_prefill", op="select", b=4, hkv=8, gqa=4, length=131072, ragged=True, meta=32, keep=128,
             update=True),
        # a decode step at 128K over 64 of 1024 groups a head, and a 77-token window
        dict(name="sparse_128k", op="sparse", b=1, hkv=8, gqa=4, length=131072 - 51, ragged=False, meta=32, type="bf16",
             keep=64, empty=0.0),
        # the batch of 32 at 32K over 64 of 256 groups a head
        dict(name="sparse_b32_32k", op="sparse", b=32, hkv=8, gqa=4, length=32768, ragged=False, meta=32, type="bf16",
             keep=64, empty=0.0),
        # a ragged batch, 8 query heads a KV head, 16-bit metadata, float32 outputs, some entries left empty
        dict(name="sparse_ragged_gqa8", op="sparse", b=7, hkv=4, gqa=8, length=20011, ragged=True, meta=16, type="f32",
             keep=37, empty=0.2),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rotary", "read", "select", "sparse"])
    hkv = rng.choice([1, 2, 4, 8])
    gqa = rng.choice([1, 2, 3, 4, 5, 8])
    meta = rng.choice([32, 32, 16])
    kind = rng.choice(["bf16", "bf16", "f32"])
    ragged = rng.random() < 0.5
    if op == "rotary":
        # at most the bytes of rotary_chunk
        size = 2 if kind == "bf16" else 4
        most = 8192 * 40 * 2 // (hkv * (gqa + 1) * size)
        return dict(op=op, n=_log(rng, 1, min(most, 16384)), hq=hkv * gqa, hkv=hkv, type=kind,
                    dim=rng.choice([16, 32, 64, 96, 128]), interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "banded", "yarn"]), factor=rng.choice([2.0, 4.0, 8.0]),
                    base=rng.choice([10000.0, 500000.0]), first=rng.randrange(0, 262144), fused=rng.random() < 0.5,
                    transpose=rng.random() < 0.3)
    if op == "read":
        b = rng.randint(1, 6)
        most = 131072 * 8 // (b * hkv * (1 if kind == "bf16" else 2))
        return dict(op=op, b=b, hkv=hkv, length=_log(rng, 1, min(131072, most)), ragged=ragged, meta=meta, type=kind,
                    part=rng.random() < 0.5)
    if op == "select":
        update = rng.random() < 0.3
        b = _log(rng, 1, 32)
        most = (4 if update else 16) * 8 * 131072 // (2 * b * hkv)
        length = _log(rng, 4096, min(131072, most))
        return dict(op=op, b=b, hkv=hkv, gqa=gqa, length=length, ragged=ragged, meta=meta,
                    keep=_log(rng, 8, max(8, length // G // 2)), update=update)
    b = _log(rng, 1, 32)
    length = _log(rng, 60, min(131072, 32 * 32768 * 8 // (b * hkv)))
    keep = _log(rng, 1, max(1, min(256, 32 * 8 * 64 * 4 // (b * hkv * max(4, gqa)))))
    return dict(op=op, b=b, hkv=hkv, gqa=gqa, length=length, ragged=ragged, meta=meta, type=kind, keep=keep,
                empty=rng.choice([0.0, 0.0, 0.3]))


def _lengths(case):
    """Tokens of each sequence: all `length`, or spread below it (the first one whole), odd ones among them."""
    if not case["ragged"]:
        return [case["length"]] * case["b"]
    n, b = case["length"], case["b"]
    return [max(1, n - (i * n) // b - 13 * i) for i in range(b)]


def _ranges(case):
    """Token ranges to read of each sequence: all of it, or a part that starts and ends anywhere."""
    out = []
    for i, n in enumerate(_lengths(case)):
        if case["part"]:
            lo = min(n - 1, n // 7 + 5 * i)
            out.append((lo, max(lo, n - n // 11 - i)))
        else:
            out.append((0, n))
    return out


def work(case):
    op = case["op"]
    if op == "rotary":
        size = 2 if case["type"] == "bf16" else 4
        rows = case["n"] * (case["hq"] + case["hkv"])
        return {"bytes": rows * D * size * 2 + 4 * case["n"], "flops": rows * (case["dim"] // 2) * 6}
    lens, hkv = _lengths(case), case["hkv"]
    block = 13824 if case["meta"] == 32 else 11008
    if op == "read":
        size = 2 if case["type"] == "bf16" else 4
        packed = sum(max(0, min(e, n // G * G) - s) for (s, e), n in zip(_ranges(case), lens))
        rows = sum(e - s for s, e in _ranges(case))
        return {"bytes": hkv * (packed * block // G + (rows - packed) * 4 * D + rows * 2 * D * size),
                "flops": hkv * packed * (2 * D + 8 * D + 2 * D)}
    hq, groups = hkv * case["gqa"], sum(n // G for n in lens)
    if op == "select":
        params = (1536 if case["meta"] == 32 else 768) + 264 if case["update"] else 264
        return {"bytes": hkv * groups * params + case["b"] * (hq * D * 2 + hkv * case["keep"] * 4),
                "flops": hq * groups * 4 * D}
    attended = [min(case["keep"], n // G) * (1.0 - case["empty"]) for n in lens]
    window = sum(n % G for n in lens)
    out = 2 if case["type"] == "bf16" else 4
    return {"bytes": int(hkv * (sum(attended) * block + window * 4 * D) + case["b"] * (hq * (D * (2 + out) + 4) +
                                                                                   hkv * case["keep"] * 4)),
            "flops": int(4 * D * hq // hkv * hkv * (sum(attended) * G + window))}


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


def _cache(case, seed):
    """A batch's packed groups [b, hkv, groups, block], windows [b, hkv, 2, 128, 128] and value maxima [b, 2, hkv]."""
    dev, lens, hkv = _device(), _lengths(case), case["hkv"]
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
    return lens, raw, window, top.transpose(1, 2).contiguous()


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


def _summaries(raw, meta):
    """8-bit range of each group's keys: lowest and highest value of every channel in steps of 2^e, and 2^e times
    the largest and the smallest norm."""
    t, at = (torch.float32, (4096, 4608, 5120, 5632)) if meta == 32 else (torch.float16, (4096, 4352, 4608, 4864))
    part = lambda i: raw[..., at[i]:at[i + 1]].contiguous().view(t).float()  # noqa: E731
    s, lo, norm = part(0), part(1), part(2)
    hi = (lo.double() + 3.0 * s.double()).float()
    top = torch.maximum(lo.abs(), hi.abs()).amax(-1, keepdim=True) if raw.numel() else lo[..., :1]
    m, x = torch.frexp(top)
    e = torch.where(m <= 127.0 / 128.0, x - 7, x - 6)
    e = torch.where(top > 0, e, torch.full_like(e, -100)).clamp_min(-100)
    lo8, hi8 = torch.round(torch.ldexp(lo, -e)), torch.round(torch.ldexp(hi, -e))
    w = torch.stack([norm.amax(-1), norm.amin(-1)], -1) if raw.numel() else norm[..., :2]
    return lo8.to(torch.int8), hi8.to(torch.int8), torch.ldexp(w, e)


# ------------------------------------------------------------ rotary angles

def _frequencies(case):
    """Frequency of each rotated pair (64 bits) and the factor on the rotated values."""
    dim, base, factor, kind = case["dim"], case["base"], case["factor"], case["scaling"]
    original = 8192
    f = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
    if kind == "none":
        return f, 1.0
    if kind == "linear":
        return [x / factor for x in f], 1.0
    if kind == "banded":
        # short wavelengths stay, long ones stretch, a ramp between
        low, high = 1.0, 4.0
        out = []
        for x in f:
            turns = original * x / (2.0 * math.pi)
            ramp = min(1.0, max(0.0, (turns - low) / (high - low)))
            out.append((1.0 - ramp) * x / factor + ramp * x)
        return out, 1.0
    # yarn: the ramp runs over the pair's index
    fast, slow = 32.0, 1.0
    at = lambda turns: dim * math.log(original / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))  # noqa: E731
    low, high = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), dim - 1)
    high = high + 0.001 if low == high else high
    ramp = [min(1.0, max(0.0, (i - low) / (high - low))) for i in range(dim // 2)]
    return [x / factor * r + x * (1.0 - r) for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0


# ------------------------------------------------------- inputs of each case

def prepare(case, seed):
    return {"rotary": _prepare_rotary, "read": _prepare_read, "select": _prepare_select,
            "sparse": _prepare_sparse}[case["op"]](case, seed)


def _rotary_inputs(case, seed):
    dev, gen, n, hq, hkv = _device(), _gen(seed, 2), case["n"], case["hq"], case["hkv"]
    heads = hq + 2 * hkv if case["fused"] else hq
    x = torch.randn((n, heads, D), device=dev, generator=gen).to(_dtype(case))
    # a fused projection's rows hold q, k and v side by side
    k = x[:, hq:hq + hkv] if case["fused"] else torch.randn((n, hkv, D), device=dev, generator=gen).to(_dtype(case))
    pos = (case["first"] + torch.arange(n, device=dev)).to(torch.int32)
    return x[:, :hq], k, pos


def _prepare_rotary(case, seed):
    q, k, pos = _rotary_inputs(case, seed)
    f, m = _frequencies(case)
    st = dict(case=case, q=q, k=k, pos=pos)
    if own:
        from int2_kv_cache_oscar_gb300 import oscar as O
        st["O"] = O
        st["config"] = O.make_rotary_config(case["dim"], base=case["base"], interleaved=case["interleaved"],
                                            scaling=case["scaling"], factor=case["factor"], original_length=8192)
        st["q_out"], st["k_out"] = torch.empty(q.shape, dtype=q.dtype, device=q.device), \
            torch.empty(k.shape, dtype=k.dtype, device=k.device)
    else:
        st["freq"], st["factor"] = torch.tensor(f, dtype=torch.float64, device=q.device), m
    return st


def _own_cache(case, lens, raw, window, top):
    from int2_kv_cache_oscar_gb300 import oscar as O
    cache = O.OscarCache(len(lens), case["hkv"], max(lens), meta_bits=case["meta"])
    for i, n in enumerate(lens):
        cache.import_sequence(i, n, raw[i, :, :n // G].contiguous(), window[i], top[i])
    return O, cache


def _prepare_read(case, seed):
    lens, raw, window, top = _cache(case, seed)
    ranges = _ranges(case)
    st = dict(case=case, ids=list(range(len(lens))), start=[a for a, _ in ranges], end=[e for _, e in ranges])
    rows = sum(e - a for a, e in ranges)
    if own:
        st["O"], st["cache"] = _own_cache(case, lens, raw, window, top)
        st["k"] = torch.empty((rows, case["hkv"], D), dtype=_dtype(case), device=raw.device)
        st["v"] = torch.empty_like(st["k"])
    else:
        st["raw"], st["window"] = raw, window
        # where each row of the output lies: its sequence and its token
        st["seq"] = torch.cat([torch.full((e - a,), i, device=raw.device) for i, (a, e) in enumerate(ranges)])
        st["token"] = torch.cat([torch.arange(a, e, device=raw.device) for a, e in ranges])
        st["packed"] = torch.tensor([n // G * G for n in lens], device=raw.device)
    return st


def _queries(case, seed, b):
    return torch.randn((b, case["hkv"] * case["gqa"], D), device=_device(), generator=_gen(seed, 3)).bfloat16()


def _prepare_select(case, seed):
    lens, raw, window, top = _cache(case, seed)
    st = dict(case=case, ids=list(range(len(lens))), q=_queries(case, seed, len(lens)))
    if own:
        st["O"], st["cache"] = _own_cache(case, lens, raw, window, top)
        st["cache"].enable_index()
        st["cache"].update_index(st["ids"])
        st["out"] = torch.empty((len(lens), case["hkv"], case["keep"]), dtype=torch.int32, device=raw.device)
    else:
        st["groups"] = torch.tensor([n // G for n in lens], device=raw.device)
        if case["update"]:
            st["raw"] = raw
        else:
            st["index"] = _summaries(raw, case["meta"])
    return st


def _chosen(case, seed, lens):
    """Listed groups of every (sequence, KV head): distinct, ascending, -1 where an entry is empty."""
    dev, gen, b, keep = _device(), _gen(seed, 4), len(lens), case["keep"]
    ng = max(lens) // G
    if ng == 0:
        return torch.full((b, case["hkv"], keep), -1, dtype=torch.int32, device=dev)
    have = torch.tensor([n // G for n in lens], device=dev)[:, None, None]
    key = torch.rand((b, case["hkv"], ng), device=dev, generator=gen)
    key = torch.where(torch.arange(ng, device=dev) < have, key, torch.full_like(key, 2.0))
    key, at = key.sort(-1)
    at = torch.where(key < 2.0, at, torch.full_like(at, 1 << 30))[..., :keep]
    drop = torch.rand(at.shape, device=dev, generator=gen) < case["empty"]
    at = torch.where(drop, torch.full_like(at, 1 << 30), at).sort(-1).values
    at = torch.where(at == 1 << 30, torch.full_like(at, -1), at)
    return torch.nn.functional.pad(at, (0, keep - at.shape[-1]), value=-1).to(torch.int32).contiguous()


def _prepare_sparse(case, seed):
    lens, raw, window, top = _cache(case, seed)
    st = dict(case=case, ids=list(range(len(lens))), q=_queries(case, seed, len(lens)),
              groups=_chosen(case, seed, lens))
    if own:
        st["O"], st["cache"] = _own_cache(case, lens, raw, window, top)
        st["out"] = torch.empty(st["q"].shape, dtype=_dtype(case), device=raw.device)
        st["lse"] = torch.empty(st["q"].shape[:2], dtype=torch.float32, device=raw.device)
        st["workspace"] = st["cache"].workspace(len(lens), st["q"].shape[1])
    else:
        st["raw"], st["window"] = raw, window
        st["tail"] = torch.tensor([n % G for n in lens], device=raw.device)
    return st


# --------------------------------------------------------------- one pass

def run(state):
    return {"rotary": _run_rotary, "read": _run_read, "select": _run_select, "sparse": _run_sparse}[state["case"]["op"]](state)


def _turn(x, c, s, case):
    """Rotates the pairs of x [n, heads, 128] by the angles whose cosine and sine are c and s [n, 1, pairs]."""
    x, half = x.float(), case["dim"] // 2
    r, rest = x[..., :case["dim"]], x[..., case["dim"]:]
    if case["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        r = torch.cat([a * c - b * s, a * s + b * c], -1)
    return torch.cat([r, rest], -1).to(_dtype(case))


def _run_rotary(st):
    case = st["case"]
    if own:
        st["O"].oscar_rotary(st["config"], st["pos"], st["q"], st["k"], st["q_out"], st["k_out"],
                             transpose=case["transpose"])
        return {"q": st["q_out"], "k": st["k_out"]}
    angle = st["pos"].double()[:, None] * st["freq"]
    c = (torch.cos(angle) * st["factor"]).float()[:, None]
    s = (torch.sin(angle) * (-st["factor"] if case["transpose"] else st["factor"])).float()[:, None]
    return {"q": _turn(st["q"], c, s, case), "k": _turn(st["k"], c, s, case)}


def _run_read(st):
    case = st["case"]
    if own:
        st["cache"].read(st["ids"], st["start"], st["end"], st["k"], st["v"])
        return {"k": st["k"], "v": st["v"]}
    k, v = _split(st["raw"], case["meta"])                                 # [b, hkv, groups, 128, 128]
    k = k @ (_hadamard(torch.float32, k.device) / math.sqrt(D))            # the matrix is its own inverse
    k, v = k.flatten(2, 3).transpose(1, 2), v.flatten(2, 3).transpose(1, 2)    # [b, tokens, hkv, 128]
    seq, token, packed = st["seq"], st["token"], st["packed"][st["seq"]]
    in_window = (token >= packed)[:, None, None]
    w = st["window"][seq, :, :, token % G].float()                         # [rows, hkv, 2, 128]
    if k.shape[1] == 0:
        return {"k": w[:, :, 0].to(_dtype(case)), "v": w[:, :, 1].to(_dtype(case))}
    at = torch.minimum(token, (packed - 1).clamp_min(0))
    return {"k": torch.where(in_window, w[:, :, 0], k[seq, at]).to(_dtype(case)),
            "v": torch.where(in_window, w[:, :, 1], v[seq, at]).to(_dtype(case))}


def _query_bytes(q, hkv):
    """Queries [b, hq, 128] -> 8-bit rotated queries [b, hkv, gqa, 128], one step size for the heads of a KV head."""
    x = q.double().unflatten(1, (hkv, -1))
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    top = x.abs().amax((2, 3), keepdim=True)
    e = torch.frexp(top)[1].clamp_min(-100)
    a = torch.round(torch.ldexp(x, 22 - e))                                # whole numbers of at most 23 bits
    r = (a @ _hadamard(torch.float64, q.device)).long()                    # whole numbers: exact
    top = r.abs().amax((2, 3), keepdim=True)
    shift = (top > (127 << torch.arange(31, device=q.device))).sum(-1, keepdim=True)
    return ((r + ((1 << shift) >> 1)) >> shift).float()


def _run_select(st):
    case = st["case"]
    if own:
        if case["update"]:
            st["cache"].update_index(st["ids"], rebuild=True)
        st["cache"].select_groups(st["ids"], st["q"], st["q"].shape[1], st["out"], keep_first=1, keep_last=1)
        return st["out"]
    q8, keep, have = _query_bytes(st["q"], case["hkv"]), case["keep"], st["groups"][:, None, None]
    lo8, hi8, w = _summaries(st["raw"], case["meta"]) if case["update"] else st["index"]
    ng = w.shape[2]
    if ng == 0:
        return torch.full((q8.shape[0], case["hkv"], keep), -1, dtype=torch.int32, device=w.device)
    # sum over the channels of max(q lo, q hi): whole numbers below 2^22, exact in 32 bits
    s = q8.clamp_min(0) @ hi8.float().transpose(-1, -2) + q8.clamp_max(0) @ lo8.float().transpose(-1, -2)
    s = s.amax(2).double()
    est = s * torch.where(s >= 0, w[..., 0], w[..., 1]).double()           # 22 x 24 bits: exact in 64
    at = torch.arange(ng, device=w.device)
    est = torch.where((at == 0) | (at == have - 1), torch.full_like(est, math.inf), est)
    est = torch.where(at < have, est, torch.full_like(est, -math.inf))
    top = torch.sort(est, dim=-1, descending=True, stable=True).indices[..., :keep]
    top = torch.where(top < have, top, torch.full_like(top, ng)).sort(-1).values
    top = torch.where(top < ng, top, torch.full_like(top, -1))
    return torch.nn.functional.pad(top, (0, keep - top.shape[-1]), value=-1).to(torch.int32)


def _run_sparse(st):
    case = st["case"]
    if own:
        st["cache"].sparse_decode(st["ids"], st["q"], st["q"].shape[1], st["groups"], st["out"], st["workspace"],
                                  lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    raw, idx, hkv = st["raw"], st["groups"].long(), case["hkv"]
    b, keep = idx.shape[0], idx.shape[2]
    q = st["q"].float().unflatten(1, (hkv, -1))                            # [b, hkv, gqa, 128]
    scale = 1.0 / math.sqrt(D)
    s_w = q @ st["window"][:, :, 0].float().transpose(-1, -2) * scale      # window: [b, hkv, gqa, 128]
    no = torch.arange(G, device=q.device) >= st["tail"][:, None, None, None]
    scores, values = s_w.masked_fill(no, -math.inf), st["window"][:, :, 1].float()
    if raw.shape[2]:
        at = (torch.arange(b, device=q.device)[:, None, None], torch.arange(hkv, device=q.device)[:, None])
        k, v = _split(raw[at[0], at[1], idx.clamp_min(0)], case["meta"])   # [b, hkv, keep, 128, 128]
        q_rot = q @ (_hadamard(torch.float32, q.device) / math.sqrt(D))
        s = q_rot @ k.flatten(2, 3).transpose(-1, -2) * scale
        s = s.masked_fill((idx < 0).repeat_interleave(G, -1)[:, :, None], -math.inf)
        scores, values = torch.cat([s, scores], -1), torch.cat([v.flatten(2, 3), values], 2)
    m = scores.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(scores - m0)
    l = p.sum(-1, keepdim=True)
    o = (p @ values) / torch.where(l > 0, l, torch.ones_like(l))
    return {"out": o.flatten(1, 2).to(_dtype(case)), "lse": (m0 + torch.log(l)).squeeze(-1).flatten(1, 2)}


# ------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    return {"rotary": _exact_rotary, "read": _exact_read, "select": _exact_select, "sparse": _exact_sparse}[case["op"]](case, seed)


def _exact_rotary(case, seed):
    q, k, pos = _rotary_inputs(case, seed)
    f, m = _frequencies(case)
    turn = -1.0 if case["transpose"] else 1.0
    wave = torch.polar(torch.full((len(f),), float(m), dtype=torch.float64, device=q.device)[None].expand(case["n"], -1).contiguous(),
                       turn * pos.double()[:, None] * torch.tensor(f, dtype=torch.float64, device=q.device))[:, None]
    out = {}
    for name, x in (("q", q), ("k", k)):
        y = x.double().clone()
        if case["interleaved"]:
            first, second = slice(0, case["dim"], 2), slice(1, case["dim"], 2)
        else:
            first, second = slice(0, case["dim"] // 2), slice(case["dim"] // 2, case["dim"])
        z = torch.complex(y[..., first], y[..., second]) * wave
        y[..., first], y[..., second] = z.real, z.imag
        out[name] = y
    return out


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


def _exact_read(case, seed):
    lens, raw, window, _ = _cache(case, seed)
    h = _hadamard(torch.float64, raw.device)
    ks, vs = [], []
    for i, (a, e) in enumerate(_ranges(case)):
        ng = lens[i] // G
        kr = torch.empty((e - a, case["hkv"], D), dtype=torch.float64, device=raw.device)
        vr = torch.empty_like(kr)
        for j in range(case["hkv"]):
            kj = torch.empty((lens[i], D), dtype=torch.float64, device=raw.device)
            vj = torch.empty_like(kj)
            for c in range(0, ng, 256):
                m = min(256, ng - c)
                k, v = _exact_blocks(raw[i, j, c:c + m], case["meta"])
                kj[c * G:(c + m) * G] = (k.view(-1, D) @ h) / math.sqrt(D)
                vj[c * G:(c + m) * G] = v.view(-1, D)
            kj[ng * G:], vj[ng * G:] = window[i, j, 0, :lens[i] % G].double(), window[i, j, 1, :lens[i] % G].double()
            kr[:, j], vr[:, j] = kj[a:e], vj[a:e]
        ks.append(kr)
        vs.append(vr)
    return {"k": torch.cat(ks), "v": torch.cat(vs)}


def _exact_select(case, seed):
    lens, raw, _, _ = _cache(case, seed)
    q, hkv, gqa, keep = _queries(case, seed, len(lens)).double().cpu(), case["hkv"], case["gqa"], case["keep"]
    wide = case["meta"] == 32
    head = raw[..., 4096:5632 if wide else 4864].contiguous().view(torch.float32 if wide else torch.float16).double().cpu()
    h = _hadamard(torch.float64, "cpu")
    out = torch.full((len(lens), hkv, keep), -1, dtype=torch.int32)
    for i, n in enumerate(lens):
        ng = n // G
        for j in range(hkv if ng else 0):
            rows = q[i, j * gqa:(j + 1) * gqa]
            e = max(math.frexp(float(rows.abs().max()))[1], -100)
            turned = torch.round(rows * 2.0 ** (22 - e)) @ h
            step = 1.0
            while float(turned.abs().max()) > 127 * step:
                step *= 2.0
            q8 = torch.floor(turned / step + (0.5 if step > 1 else 0.0))
            s, z, norm = head[i, j, :ng].unflatten(-1, (3, D)).unbind(-2)
            up = (z + 3 * s).float().double()
            top = torch.maximum(z.abs(), up.abs()).amax(-1)
            unit = torch.tensor([2.0 ** max(math.ceil(math.log2(float(t) / 127 * (1 - 1e-12))), -100) if t > 0 else 2.0 ** -100 for t in top],
                                dtype=torch.float64)
            unit = torch.where(127 * unit >= top, unit, 2 * unit)
            low, high = torch.round(z / unit[:, None]), torch.round(up / unit[:, None])
            s = torch.stack([torch.maximum(x * low, x * high).sum(-1) for x in q8]).amax(0)
            est = s * torch.where(s >= 0, norm.amax(-1), norm.amin(-1)) * unit
            est[0] = est[ng - 1] = math.inf
            order = sorted(range(ng), key=lambda t: (-float(est[t]), t))[:keep]
            out[i, j, :len(order)] = torch.tensor(sorted(order), dtype=torch.int32)
    return out.to(raw.device)


def _exact_sparse(case, seed):
    lens, raw, window, _ = _cache(case, seed)
    q, groups, hkv, gqa = _queries(case, seed, len(lens)).double(), _chosen(case, seed, lens), case["hkv"], case["gqa"]
    h = _hadamard(torch.float64, raw.device)
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=raw.device)
    for i, n in enumerate(lens):
        for j in range(hkv):
            idx = groups[i, j][groups[i, j] >= 0].long()
            k, v = window[i, j, 0, :n % G].double(), window[i, j, 1, :n % G].double()
            if idx.numel():
                kq, vq = _exact_blocks(raw[i, j, idx], case["meta"])
                k = torch.cat([(kq.view(-1, D) @ h) / math.sqrt(D), k])
                v = torch.cat([vq.view(-1, D), v])
            if k.shape[0] == 0:
                continue
            s = q[i, j * gqa:(j + 1) * gqa] @ k.T / math.sqrt(D)
            lse[i, j * gqa:(j + 1) * gqa] = torch.logsumexp(s, -1)
            out[i, j * gqa:(j + 1) * gqa] = torch.softmax(s, -1) @ v
    return {"out": out, "lse": lse}
