"""Measured cases of the operators that bring a prompt in and draw tokens.

A program that answers prompts appends a prompt's keys and values to the paged
8-bit cache, rotated on the way, lets the rows that answer it share its pages,
rotates a step's queries and keys, and draws tokens from logits that top-k,
top-p and min-p cut.  Each case is one call of one of these:

  sample    tokens drawn from [B, P, V] logits by given uniforms
  truncate  the logits that top-k, top-p and min-p cut become -inf
  rotate    a step's queries and keys are rotated by their positions
  append    a prompt's keys and values into the cache, keys rotated on the way
  prefix    attention of a step's tokens over a prefix that rows share, their
            own cache and each other

With ``own`` false, ``run`` computes the plain form in elementary torch
operations; with ``own`` true it makes the framework's calls.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
LARGEST_LOGITS = 256 * 201088 * 2       # bytes of the largest listed logits
LARGEST_TOKENS = 16 * 4096              # tokens x (H + 2 Hkv) of 48 of the largest append or rotation
LARGEST_SCORES = 64 * 6 * 32 * 8192     # scores of the largest listed prefix
LARGEST_KEYS = 64 * 8192 * 8 * 128      # values of the prefix's keys, were they one copy per row


# ---- cases ----------------------------------------------------------------------

def _sample(name, B, P, V, dtype, n, controls, op="sample", T=0.8, greedy=0, ld=0):
    """n: draws per position; controls: which of k, p and m (top-k, top-p, min-p) are given; T: the rows' temperature,
    greedy: one row in so many is greedy (0: none); ld: the logits' row pitch (0: V)."""
    c = dict(op=op, B=B, P=P, V=V, dtype=dtype, n=n, controls=controls, T=T, greedy=greedy, ld=ld or V)
    return dict(c, name=name) if name else c


def _rotate(name, B, T, H, Hkv, D, R, ctx, tree=False, interleaved=False, axes=1, padded=False):
    """R: rotated channels; axes: numbers to a position (3: time, height, width); padded: rows hold fewer tokens."""
    c = dict(op="rotate", B=B, T=T, H=H, Hkv=Hkv, D=D, R=R, ctx=ctx, tree=tree, interleaved=interleaved, axes=axes,
             padded=padded)
    return dict(c, name=name) if name else c


def _append(name, B, T, Hkv, D, R, page, kind, ctx, interleaved=False, axes=1, keys=False):
    """T: the longest prompt; ctx: what the longest row held before; keys: the rotated keys come back too."""
    c = dict(op="append", B=B, T=T, Hkv=Hkv, D=D, R=R, page=page, kind=kind, ctx=ctx, interleaved=interleaved,
             axes=axes, keys=keys)
    return dict(c, name=name) if name else c


def _prefix(name, B, T, H, Hkv, D, page, kind, prefix, groups, ctx, tree=False, weights=False, padded=False):
    """prefix: tokens of the longest shared prefix; groups: prefixes in the batch; ctx: the longest row's own tokens
    past it."""
    c = dict(op="prefix", B=B, T=T, H=H, Hkv=Hkv, D=D, page=page, kind=kind, prefix=prefix, groups=groups, ctx=ctx,
             tree=tree, weights=weights, padded=padded)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one interactive user's next token under every control: the latency of a call
        _sample("sample-one-token", 1, 1, 128256, "bf16", 1, "kpm"),
        # a full batch's next tokens over the largest vocabulary, nucleus sampling, one row in eight greedy
        _sample("sample-nucleus-batch", 256, 1, 201088, "bf16", 1, "pm", greedy=8),
        # drafts of trees: four siblings of each of 13 nodes, top-k drafts in float32 over an odd vocabulary
        _sample("sample-siblings-f32-odd", 24, 13, 32003, "f32", 4, "k", T=1.0),
        # one user's target logits of a chain of five drafts, cut before they are verified
        _sample("truncate-one-chain", 1, 6, 128256, "bf16", 0, "p", op="truncate"),
        # a batch's target logits at the framework's config-1 shape
        _sample("truncate-chains", 64, 6, 151936, "bf16", 0, "kp", op="truncate", T=0.6),
        # one user's token
        _rotate("rotate-one-token", 1, 1, 32, 8, 128, 128, 987),
        # the 61-node tree workload, padded trees, far positions
        _rotate("rotate-trees", 32, 61, 32, 8, 128, 128, 131072, tree=True, padded=True),
        # one user's prompt of odd length after an earlier turn
        _append("append-one-prompt", 1, 1001, 8, 128, 128, 64, "e4m3", 345),
        # a batch of prompts with pictures (positions of three axes), the rotated keys for the prompt's own attention
        _append("append-prompts", 16, 4096, 8, 128, 128, 64, "e4m3", 0, axes=3, keys=True),
        # eight answers to one document, plain decoding
        _prefix("prefix-few-rows", 8, 1, 32, 8, 128, 64, "e4m3", 8192, 1, 300),
        # many answers to one long prompt, chains of five drafts
        _prefix("prefix-chains", 64, 6, 32, 8, 128, 64, "e4m3", 8192, 1, 512),
        # trees under four system prompts, int8, small pages, block weights for eviction
        _prefix("prefix-trees-int8-groups", 32, 61, 32, 8, 64, 16, "int8", 2048, 4, 700, tree=True, weights=True,
                padded=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["sample", "sample", "truncate", "rotate", "append", "prefix", "prefix"])
    if op in ("sample", "truncate"):
        dtype = rng.choice(["bf16", "f32"])
        V, P = _log(rng, 1000, 202000), rng.randint(1, 16)
        most = LARGEST_LOGITS // (P * V * (2 if dtype == "bf16" else 4))
        controls = rng.choice(["k", "p", "m", "kp", "pm", "kpm"] + ([""] if op == "sample" else []))
        return _sample("", _log(rng, 1, max(1, min(256, most))), P, V, dtype,
                       rng.choice([1, 1, rng.randint(2, 8)]) if op == "sample" else 0, controls, op,
                       rng.choice([0.6, 0.8, 1.0]), rng.choice([0, 0, 4]), V + rng.choice([0, 0, rng.randint(1, 64)]))
    H, Hkv = rng.choice([(32, 8), (64, 8), (16, 16), (28, 4), (40, 8), (8, 1), (6, 2)])
    D = rng.choice([64, 128])
    tree = rng.random() < 0.3
    if op == "rotate":
        T = rng.randint(2, 64) if tree else _log(rng, 1, 2048)
        axes = 1 if tree else rng.choice([1, 1, 3])
        return _rotate("", _log(rng, 1, max(1, min(256, LARGEST_TOKENS * 48 // (T * (H + Hkv) * 2)))), T, H, Hkv, D,
                       rng.choice([D, D, D // 2]), _log(rng, 1, 131072), tree, rng.random() < 0.3, axes,
                       rng.random() < 0.4)
    page, kind = rng.choice([16, 32, 64, 128]), rng.choice(["e4m3", "int8"])
    if op == "append":
        T = _log(rng, 1, 8192)
        return _append("", _log(rng, 1, max(1, min(64, LARGEST_TOKENS * 8 // (T * Hkv)))), T, Hkv, D,
                       rng.choice([0, D, D, D // 2]), page, kind, _log(rng, 1, 8192), rng.random() < 0.3,
                       rng.choice([1, 1, 3]), rng.random() < 0.4)
    T = rng.randint(2, 64) if tree else rng.randint(1, 10)
    prefix = _log(rng, 16, 32768)
    most = min(LARGEST_SCORES // (T * H * prefix), LARGEST_KEYS // (prefix * Hkv * D))
    B = _log(rng, 1, max(1, min(64, most)))
    return _prefix("", B, T, H, Hkv, D, page, kind, prefix, rng.randint(1, min(B, 4)), _log(rng, 1, 1024), tree,
                   rng.random() < 0.3, rng.random() < 0.3)


# ---- what a case's rows hold (rules of the row's number, so that work() can count them) ---------

def _frac(b, salt=0.0):
    return (0.5 + 0.6180339887498949 * b + salt) % 1.0


def _contexts(c):
    """Tokens that each row held before: the first row's are ctx, the others' spread over an eighth of it and more."""
    return [c["ctx"]] + [int(c["ctx"] * (0.125 + 0.875 * _frac(b))) for b in range(1, c["B"])]


def _queries(c):
    if not c.get("padded"):
        return [c["T"]] * c["B"]
    return [max(1, int(c["T"] * (0.5 + 0.5 * _frac(b, 0.3)) + 0.5)) for b in range(c["B"])]


def _prompts(c):
    """New tokens of each row of an append."""
    return [c["T"]] + [max(1, int(c["T"] * (0.25 + 0.75 * _frac(b, 0.1)))) for b in range(1, c["B"])]


def _group_starts(c):
    """Row prefix_starts[g] is the first that begins with prefix g; the last row of a batch of several goes without."""
    rows = c["B"] - (1 if c["groups"] > 1 and c["B"] > c["groups"] else 0)
    return [rows * g // c["groups"] for g in range(c["groups"] + 1)]


def _prefix_blocks(c):
    most = max(1, c["prefix"] // c["page"])
    return [most] + [max(1, int(most * (0.5 + 0.5 * _frac(g)))) for g in range(1, c["groups"])]


# ---- inputs ------------------------------------------------------------------------

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _parents(g, B, N):
    """Random trees: the parent of node c is one of the four nodes before it."""
    r = torch.rand((B, N), generator=g, device=DEV)
    c = torch.arange(N, device=DEV)
    back = torch.minimum(c, torch.full_like(c, 4))
    return (c - 1 - (r * back).floor()).clamp(min=0).to(torch.int32).contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return {"sample": _prepare_sample, "truncate": _prepare_sample, "rotate": _prepare_rotate,
            "append": _prepare_append, "prefix": _prepare_prefix}[case["op"]](case, g)


def _prepare_sample(c, g):
    B, P, V, ld = c["B"], c["P"], c["V"], c["ld"]
    dt = BF16 if c["dtype"] == "bf16" else F32
    store = torch.empty((B, P, ld), dtype=dt, device=DEV)
    peaks = torch.randint(0, V, (B, P, 20), generator=g, device=DEV)
    for b in range(B):  # as the verifier's workloads: a normal base and 20 tokens that stand out
        x = torch.randn((P, ld), generator=g, device=DEV) * 3
        store[b] = x.scatter_add_(1, peaks[b], torch.full((P, 20), 8.0, device=DEV)).to(dt)
    s = dict(c=c, logits=store[:, :, :V])
    t = torch.full((B,), c["T"], device=DEV)
    if c["greedy"]:
        t[c["greedy"] - 1::c["greedy"]] = 0.0
    s["temperature"] = t
    s["uniforms"] = torch.rand((B, P, max(1, c["n"])), generator=g, device=DEV)
    # requests differ; one row in nine has a control left off
    u = torch.rand((3, B), generator=g, device=DEV)
    off = torch.arange(B, device=DEV) % 9 == 8
    k = torch.exp(math.log(10) + u[0] * math.log(12.8)).round().to(torch.int32)  # 10 .. 128
    s["top_k"] = torch.where(off, 0, k).to(torch.int32) if "k" in c["controls"] else None
    s["top_p"] = torch.where(off, 1.0, 0.8 + 0.19 * u[1]) if "p" in c["controls"] else None
    s["min_p"] = torch.where(off, 0.0, 0.02 + 0.1 * u[2]) if "m" in c["controls"] else None
    return s


def _freqs(R):
    """Rotary frequencies per token: powers of a base, as models have them."""
    return (500000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R)).to(F32)


def _positions_of_pictures(g, axes, B, T, start):
    """Positions of several axes: runs of text count on all axes at once, pictures go by row and column."""
    t = torch.arange(T, device=DEV)[None, :] + start[:, None]
    ids = t[None].expand(axes, B, T).clone()
    at = (t // 100) % 3 == 1  # every third hundred of tokens is a picture of rows of 10
    for a in range(1, axes):
        inside = t % 100
        ids[a] = torch.where(at, t - inside + (inside // 10 if a == 1 else inside % 10), t)
    ids[0] = torch.where(at, t - t % 100, t)
    return ids.to(torch.int32).contiguous()


def _rotary(c, g, s, start):
    R = c["R"]
    s["freqs"] = _freqs(R) if R else None
    s["ids"] = s["axes"] = None
    if R and c["axes"] > 1:
        s["ids"] = _positions_of_pictures(g, c["axes"], c["B"], c["T"], start)
        # a half of the pairs goes by the first axis, a quarter by each of the others
        i = torch.arange(R // 2, device=DEV)
        s["axes"] = torch.where(i < R // 4, 0, torch.where(i < 3 * R // 8, 1, 2)).clamp(max=c["axes"] - 1).to(torch.int32)


def _prepare_rotate(c, g):
    B, T, H, Hkv, D = (c[k] for k in ("B", "T", "H", "Hkv", "D"))
    s = dict(c=c)
    qkv = torch.empty((B, T, H + 2 * Hkv, D), dtype=BF16, device=DEV)  # one projection's output
    for b in range(B):
        qkv[b] = torch.randn((T, H + 2 * Hkv, D), generator=g, device=DEV).to(BF16)
    s["q"], s["k"] = qkv[:, :, :H], qkv[:, :, H:H + Hkv]
    s["positions"] = _ints(_contexts(c))
    s["parents"] = _parents(g, B, T) if c["tree"] else None
    s["query_lens"] = _ints(_queries(c)) if c["padded"] else None
    s["q_out"] = torch.zeros((B, T, H, D), dtype=BF16, device=DEV)
    s["k_out"] = torch.zeros((B, T, Hkv, D), dtype=BF16, device=DEV)
    _rotary(c, g, s, s["positions"])
    return s


def _ring_pages(c, ctx, new):
    """A tail in which no row's new tokens lie where its old ones were, so that a pass leaves its own input as it was."""
    page, n = c["page"], 2
    while any(x % page and (x % page + t) // page and (x % page + t) // page % n == 0 for x, t in zip(ctx, new)):
        n += 1
    return n


def _prepare_append(c, g):
    B, T, Hkv, D, page = (c[k] for k in ("B", "T", "Hkv", "D", "page"))
    ctx, new = _contexts(c), _prompts(c)
    blocks = [x // page for x in ctx]
    reserve = [(x % page + t) // page for x, t in zip(ctx, new)]
    most = max(x + r for x, r in zip(blocks, reserve)) + 1
    pages = max(1, sum(reserve))  # only the reserve's pages are written, so the pool holds no others
    s = dict(c=c)
    s["k_pages"] = torch.zeros((pages, Hkv, page, D), dtype=torch.uint8, device=DEV)
    s["v_pages"] = torch.zeros((pages, Hkv, D, page), dtype=torch.uint8, device=DEV)
    s["k_scale"], s["v_scale"] = (torch.ones((pages, Hkv), device=DEV) for _ in range(2))
    gain = torch.exp(torch.randn((Hkv, D), generator=g, device=DEV) * 0.7)  # channels differ, as keys' do
    ring = _ring_pages(c, ctx, new) * page
    for k in ("k_tail", "v_tail"):
        s[k] = (torch.randn((B, ring, Hkv, D), generator=g, device=DEV) * gain).to(BF16)
    kv = torch.empty((B, T, 2, Hkv, D), dtype=BF16, device=DEV)
    for b in range(B):
        kv[b] = (torch.randn((T, 2, Hkv, D), generator=g, device=DEV) * gain).to(BF16)
    s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    s["table"] = torch.full((B, most), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b in range(B):
        s["table"][b, blocks[b]:blocks[b] + reserve[b]] = perm[at:at + reserve[b]]
        at += reserve[b]
    s["positions"], s["blocks"], s["lens"] = _ints(ctx), _ints(blocks), _ints(new)
    s["k_out"] = torch.zeros((B, T, Hkv, D), dtype=BF16, device=DEV) if c["keys"] else None
    _rotary(c, g, s, s["positions"])
    return s


def _codes(g, shape, kind):
    """Cached values as a quantiser leaves them: normal values with the block's largest at the end of the range."""
    x = torch.randn(shape, generator=g, device=DEV)
    return ((x * 28).round().clamp(-127, 127).to(torch.int8).view(torch.uint8) if kind == "int8"
            else (x * 90).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))


def _prepare_prefix(c, g):
    B, T, H, Hkv, D, page = (c[k] for k in ("B", "T", "H", "Hkv", "D", "page"))
    starts, shared = _group_starts(c), _prefix_blocks(c)
    of = [next((i for i in range(c["groups"]) if starts[i] <= b < starts[i + 1]), -1) for b in range(B)]
    own_tokens = _contexts(c)
    ctx = [x + (shared[i] * page if i >= 0 else 0) for x, i in zip(own_tokens, of)]
    blocks = [x // page for x in own_tokens]
    most, pages = max(blocks) + 1, sum(blocks) + sum(shared) + B
    s = dict(c=c)
    s["k_pages"] = _codes(g, (pages, Hkv, page, D), c["kind"])
    s["v_pages"] = _codes(g, (pages, Hkv, D, page), c["kind"])
    unit = 1 / 28 if c["kind"] == "int8" else 1 / 90
    for k in ("k_scale", "v_scale"):
        s[k] = unit * (0.5 + torch.rand((pages, Hkv), generator=g, device=DEV))
    ring = -(-(page - 1 + T) // page) * page
    for k in ("k_tail", "v_tail"):
        s[k] = torch.randn((B, ring, Hkv, D), generator=g, device=DEV).to(BF16)
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    s["table"] = torch.full((B, most), -1, dtype=torch.int32, device=DEV)
    s["prefix_table"] = torch.full((c["groups"], max(shared)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b in range(B):
        n = min(most, blocks[b] + 1)
        s["table"][b, :n] = perm[at:at + n]
        at += n
    for i in range(c["groups"]):
        s["prefix_table"][i, :shared[i]] = perm[at:at + shared[i]]
        at += shared[i]
    s["positions"], s["blocks"] = _ints(ctx), _ints(blocks)
    s["prefix_blocks"], s["prefix_starts"] = _ints(shared), _ints(starts)
    s["of"] = of
    qkv = torch.randn((B, T, H + 2 * Hkv, D), generator=g, device=DEV).to(BF16)
    s["q"], s["k_new"], s["v_new"] = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
    s["parents"] = _parents(g, B, T) if c["tree"] else None
    s["query_lens"] = _ints(_queries(c)) if c["padded"] else None
    s["out"] = torch.zeros((B, T, H, D), dtype=BF16, device=DEV)
    s["weights"] = torch.zeros((B, T, most), device=DEV) if c["weights"] else None
    return s


# ---- run ----------------------------------------------------------------------------

def run(state):
    op = state["c"]["op"]
    if own:
        return {"sample": _own_sample, "truncate": _own_truncate, "rotate": _own_rotate, "append": _own_append,
                "prefix": _own_prefix}[op](state)
    return {"sample": _plain_sample, "truncate": _plain_truncate, "rotate": _plain_rotate, "append": _plain_append,
            "prefix": _plain_prefix}[op](state)


def _own_sample(s):
    import rejection_sampling_verifier_amd as rsv
    tokens, logprobs = rsv.sample_tokens(s["logits"], s["uniforms"], s["temperature"], top_k=s["top_k"],
                                         top_p=s["top_p"], min_p=s["min_p"], logprobs=True)
    return dict(tokens=tokens, logprobs=logprobs)


def _own_truncate(s):
    import rejection_sampling_verifier_amd as rsv
    return rsv.truncate_logits(s["logits"], s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])


def _own_rotate(s):
    import rejection_sampling_verifier_amd as rsv
    return rsv.rotate_tokens(s["q"], s["k"], s["freqs"], s["positions"], interleaved=s["c"]["interleaved"],
                             axes=s["axes"], ids=s["ids"], parents=s["parents"], query_lens=s["query_lens"],
                             q_out=s["q_out"], k_out=s["k_out"])


def _cache(s):
    """The handle that a user's program keeps with its cache."""
    import rejection_sampling_verifier_amd as rsv
    if "cache" not in s:
        s["cache"] = rsv.KVCache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["k_tail"], s["v_tail"],
                                 s["table"], kind=s["c"]["kind"])
    return s["cache"]


def _own_append(s):
    import rejection_sampling_verifier_amd as rsv
    positions, blocks = rsv.cache_append(_cache(s), s["k"], s["v"], s["positions"], s["blocks"], lens=s["lens"],
                                         freqs=s["freqs"], interleaved=s["c"]["interleaved"], axes=s["axes"],
                                         ids=s["ids"], k_out=s["k_out"])
    return _append_outputs(s, positions, blocks)


def _own_prefix(s):
    import rejection_sampling_verifier_amd as rsv
    return rsv.cache_attention(s["q"], s["k_new"], s["v_new"], _cache(s), s["positions"], s["blocks"],
                               parents=s["parents"], query_lens=s["query_lens"], scale=s["c"]["D"] ** -0.5,
                               prefix_table=s["prefix_table"], prefix_blocks=s["prefix_blocks"],
                               prefix_starts=s["prefix_starts"], out=s["out"], weights=s["weights"])


def _append_outputs(s, positions, blocks):
    """The pages as the values they stand for."""
    out = dict(k_scale=s["k_scale"], v_scale=s["v_scale"], k_tail=s["k_tail"], v_tail=s["v_tail"],
               positions=positions, blocks=blocks)
    for x in "kv":
        if s["c"]["kind"] == "e4m3":
            out[x + "_pages"] = s[x + "_pages"].view(torch.float8_e4m3fn)
        else:
            out[x + "_pages"] = (s[x + "_pages"].view(torch.int8) * s[x + "_scale"][:, :, None, None]).to(BF16)
    if s["k_out"] is not None:
        out["k_out"] = s["k_out"]
    return out


# ---- plain forms ----------------------------------------------------------------------

def _cut(s):
    """[R, V] truth values: what top-k, top-p and min-p leave, and the weights exp((l - max) / T) in 64 bits."""
    c = s["c"]
    R, V, P = c["B"] * c["P"], c["V"], c["P"]
    x = s["logits"].float().reshape(R, V)
    t = s["temperature"].repeat_interleave(P)[:, None].double()
    sampling = t > 0
    w = torch.exp((x.double() - x.amax(1, keepdim=True).double()) / torch.where(sampling, t, 1.0))
    if s["top_k"] is None and s["top_p"] is None and s["min_p"] is None:
        return x, w, x > -math.inf, sampling
    order = x.sort(dim=1, descending=True, stable=True).indices
    sw = w.gather(1, order)
    j = torch.arange(V, device=DEV)[None]
    live = x.gather(1, order) > -math.inf
    if s["top_k"] is not None:
        k = s["top_k"].repeat_interleave(P)[:, None]
        live &= (j < k) | (k <= 0)
    if s["top_p"] is not None:
        p = s["top_p"].repeat_interleave(P)[:, None].double()
        mass = torch.where(live, sw, 0.0).cumsum(1)
        before = torch.cat([torch.zeros_like(mass[:, :1]), mass[:, :-1]], 1)
        live &= (before < p * mass[:, -1:]) | (j == 0) | (p >= 1)
    if s["min_p"] is not None:
        live &= sw >= s["min_p"].repeat_interleave(P)[:, None].double().clamp(max=1.0)
    return x, w, torch.zeros_like(live).scatter_(1, order, live), sampling


def _plain_sample(s):
    c = s["c"]
    B, P, n = c["B"], c["P"], c["n"]
    x, w, keep, sampling = _cut(s)
    mass = torch.where(keep, w, 0.0).cumsum(1)
    total = mass[:, -1:]
    t = s["uniforms"].reshape(B * P, n).double() * total
    token = torch.searchsorted(mass, t, right=True)
    token = torch.where(sampling, token.clamp(max=c["V"] - 1), x.argmax(1, keepdim=True))
    logprob = torch.where(sampling, (w.gather(1, token) / total).log(), 0.0)
    return dict(tokens=token.view(B, P, n).int(), logprobs=logprob.float().view(B, P, n))


def _plain_truncate(s):
    c = s["c"]
    _, _, keep, sampling = _cut(s)
    keep = (keep | ~sampling).view(c["B"], c["P"], c["V"])
    return torch.where(keep, s["logits"].float(), -math.inf).to(s["logits"].dtype)


def _above(parents, B, P):
    """[B, P, P] truth values: node c is on the path root .. v, v included.  parents None: the chain."""
    eye = torch.eye(P, dtype=torch.bool, device=DEV)
    if parents is None:
        return torch.ones((P, P), dtype=torch.bool, device=DEV).tril().expand(B, P, P)
    step = torch.zeros((B, P, P), device=DEV)
    step.scatter_(2, parents.long()[:, :, None], 1.0)
    step[:, 0] = 0.0
    reach = step + eye
    for _ in range(max(1, (P - 1).bit_length())):  # paths of up to 1, 2, 4, ... steps
        reach = ((reach @ reach) > 0).float()
    return reach > 0


def _turn(x, s, ids):
    """x [B, T, heads, D] rotated by positions ids [axes, B, T], rounded to bf16."""
    R = s["c"]["R"]
    axes = s["axes"].long() if s["axes"] is not None else torch.zeros(R // 2, dtype=torch.long, device=DEV)
    angle = ids.double()[axes].permute(1, 2, 0) * s["freqs"].double()
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    x = x.float()
    if s["c"]["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., R:]], -1).to(BF16)


def _plain_rotate(s):
    c = s["c"]
    B, T = c["B"], c["T"]
    ids = s["ids"]
    if ids is None:
        depth = (_above(s["parents"], B, T).sum(2) - 1 if s["parents"] is not None
                 else torch.arange(T, device=DEV)[None].expand(B, T))
        ids = (s["positions"][:, None] + depth)[None]
    q, k = _turn(s["q"], s, ids), _turn(s["k"], s, ids)
    if s["query_lens"] is not None:
        live = (torch.arange(T, device=DEV)[None] < s["query_lens"][:, None])[:, :, None, None]
        q, k = torch.where(live, q, s["q_out"]), torch.where(live, k, s["k_out"])
    return q, k


def _scale_of(top, kind):
    """The scale of blocks with these largest magnitudes (float64 in, the float32 scale's value out)."""
    if kind == "int8":
        scale = (top / 127).float().double()
    else:
        m, e = torch.frexp(top)  # top = m 2^e with m in [0.5, 1); 448 = 0.875 * 2^9
        scale = torch.ldexp(torch.ones_like(top), e - 9 + (m > 0.875).to(e.dtype))
    return torch.where(top > 0, scale.clamp(min=2.0 ** -126), 1.0)


def _plain_append(s):
    c = s["c"]
    B, T, Hkv, D, page = (c[k] for k in ("B", "T", "Hkv", "D", "page"))
    R, most = s["k_tail"].shape[1], s["table"].shape[1]
    pos, blocks, n = s["positions"].long(), s["blocks"].long(), s["lens"].long()
    tail = pos % page
    k_new = s["k"]
    if s["freqs"] is not None:
        ids = s["ids"]
        if ids is None:
            ids = (pos[:, None] + torch.arange(T, device=DEV)[None])[None]
        k_new = _turn(s["k"], s, ids)
    if s["k_out"] is not None:
        live = (torch.arange(T, device=DEV)[None] < n[:, None])[:, :, None, None]
        s["k_out"].copy_(torch.where(live, k_new, s["k_out"]))
    filled = (tail + n) // page
    S = -(-(page - 1 + T) // page) * page
    j = torch.arange(S, device=DEV)[None].expand(B, S)
    in_tail = j < tail[:, None]
    slot = ((pos - tail)[:, None] + j) % R
    from_new = (j - tail[:, None]).clamp(0, T - 1)
    rows = torch.arange(B, device=DEV)[:, None]
    m = torch.arange(S // page, device=DEV)[None]
    done = m < filled[:, None]
    at = s["table"].long().gather(1, (blocks[:, None] + m).clamp(max=most - 1))[done]
    left = (j >= (filled * page)[:, None]) & (j >= tail[:, None]) & (j < (tail + n)[:, None])
    for x, new in (("k", k_new), ("v", s["v"])):
        seq = torch.where(in_tail[:, :, None, None], s[x + "_tail"][rows, slot], new[rows, from_new])
        blk = seq.view(B, S // page, page, Hkv, D)[done].permute(0, 2, 1, 3).float()      # [blocks, Hkv, page, D]
        scale = _scale_of(blk.abs().amax((2, 3)).double(), c["kind"])
        y = blk.double() / scale[:, :, None, None]
        code = (y.round().to(torch.int8) if c["kind"] == "int8" else y.float().to(torch.float8_e4m3fn)).view(torch.uint8)
        s[x + "_pages"][at] = code if x == "k" else code.transpose(2, 3)
        s[x + "_scale"][at] = scale.float()
        s[x + "_tail"][rows.expand(B, S)[left], slot[left]] = seq[left]
    return _append_outputs(s, (pos + n).int(), (blocks + filled).int())


def _values(codes, scale, kind):
    x = codes.view(torch.int8).float() if kind == "int8" else codes.view(torch.float8_e4m3fn).float()
    return x * scale[..., None, None]


def _cached(s, table):
    """Keys and values [rows, Hkv, blocks * page, D] of the pages of these tables."""
    c = s["c"]
    ids = table.long().clamp(min=0)
    k = _values(s["k_pages"][ids], s["k_scale"][ids], c["kind"])                       # [rows, n, Hkv, page, D]
    v = _values(s["v_pages"][ids], s["v_scale"][ids], c["kind"]).transpose(3, 4)
    return (x.permute(0, 2, 1, 3, 4).reshape(ids.shape[0], c["Hkv"], -1, c["D"]) for x in (k, v))


def _plain_prefix(s):
    c = s["c"]
    B, T, H, Hkv, D, page = (c[k] for k in ("B", "T", "H", "Hkv", "D", "page"))
    n, shared = s["table"].shape[1], s["prefix_table"].shape[1]
    k8, v8 = _cached(s, s["table"])
    kp, vp = _cached(s, s["prefix_table"])
    starts = s["prefix_starts"].long()
    row = torch.arange(B, device=DEV)
    group = torch.searchsorted(starts, row, right=True) - 1
    inside = (group >= 0) & (group < c["groups"])
    group = group.clamp(0, c["groups"] - 1)
    R = s["k_tail"].shape[1]
    pos = s["positions"].long()
    tail = pos % page
    slot = (pos - tail)[:, None] + torch.arange(page, device=DEV)[None]
    at = (slot % R)[:, :, None, None].expand(B, page, Hkv, D)
    k = torch.cat([kp[group], k8, s["k_tail"].gather(1, at).float().transpose(1, 2), s["k_new"].float().transpose(1, 2)], 2)
    v = torch.cat([vp[group], v8, s["v_tail"].gather(1, at).float().transpose(1, 2), s["v_new"].float().transpose(1, 2)], 2)
    q = s["q"].float().view(B, T, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    many = torch.where(inside, s["prefix_blocks"].long()[group], 0)
    live_p = torch.arange(shared * page, device=DEV)[None] < (many * page)[:, None]
    live8 = torch.arange(n * page, device=DEV)[None] < (s["blocks"] * page)[:, None]
    live_t = torch.arange(page, device=DEV)[None] < tail[:, None]
    see = torch.cat([torch.cat([live_p, live8, live_t], 1)[:, None].expand(B, T, -1), _above(s["parents"], B, T)], 2)
    score = torch.matmul(q, k.transpose(2, 3).contiguous()) * D ** -0.5
    score = score.view(B, Hkv, H // Hkv, T, -1).masked_fill(~see[:, None, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, Hkv, -1, p.shape[-1]), v).view(B, Hkv, H // Hkv, T, D)
    out = out.permute(0, 3, 1, 2, 4).reshape(B, T, H, D).to(BF16)
    live = None
    if s["query_lens"] is not None:
        live = torch.arange(T, device=DEV)[None] < s["query_lens"][:, None]
        out = torch.where(live[:, :, None, None], out, s["out"])
    if not c["weights"]:
        return out
    w = p[..., shared * page:(shared + n) * page].reshape(B, H, T, n, page).sum((1, 4))
    return out, w if live is None else torch.where(live[:, :, None], w, s["weights"])


# ---- work ---------------------------------------------------------------------------

def work(case):
    c = case
    B = c["B"]
    if c["op"] in ("sample", "truncate"):
        R, es = B * c["P"], 2 if c["dtype"] == "bf16" else 4
        n = R * c["V"] * es * (1 if c["op"] == "sample" else 2) + 4 * B * (1 + len(c["controls"])) + 12 * R * c["n"]
        return {"bytes": n, "flops": 2 * R * c["V"]}
    if c["op"] == "rotate":
        n = sum(_queries(c)) * (c["H"] + c["Hkv"]) * c["D"]
        return {"bytes": 4 * n + 4 * sum(_queries(c)) * (c["axes"] if c["axes"] > 1 else 0), "flops": 3 * n}
    if c["op"] == "append":
        Hkv, D, page = c["Hkv"], c["D"], c["page"]
        n = f = 0
        for x, t in zip(_contexts(c), _prompts(c)):
            tail = x % page
            filled = (tail + t) // page
            left = tail + t - filled * page if filled else t
            read = t + (tail if filled else 0)
            n += 2 * Hkv * D * (2 * read + 2 * left + filled * page) + 8 * Hkv * filled + 24
            n += 2 * Hkv * D * t if c["keys"] else 0
            f += 2 * Hkv * D * 4 * t
        return {"bytes": n, "flops": f}
    H, Hkv, D, page = (c[k] for k in ("H", "Hkv", "D", "page"))
    starts, shared = _group_starts(c), _prefix_blocks(c)
    n = sum(shared) * (2 * Hkv * D * page + 8 * Hkv + 4)
    f = 0
    for b, (x, t) in enumerate(zip(_contexts(c), _queries(c))):
        whole, tail = x // page * page, x % page
        seen = sum(shared[i] * page for i in range(c["groups"]) if starts[i] <= b < starts[i + 1])
        n += 2 * Hkv * D * (whole + 2 * tail + 2 * t) + 8 * Hkv * (whole // page) + 4 * t * H * D
        n += 4 * (whole // page) * (1 + (t if c["weights"] else 0))
        f += 4 * t * H * D * (seen + x + t)
    return {"bytes": n, "flops": f}


# ---- from the definitions, in 64 bits ----------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"sample": _exact_sample, "truncate": _exact_truncate, "rotate": _exact_rotate, "append": _exact_append,
            "prefix": _exact_prefix}[case["op"]](s)


def _host(s, *names):
    return [None if s[k] is None else s[k].cpu().numpy() for k in names]


def _kept_ids(x, t, k, p, m):
    """The tokens that the cut leaves, ascending, and their weights: one row of float64 logits."""
    order = np.lexsort((np.arange(x.size), -x))
    order = order[x[order] > -np.inf]
    if k is not None and k > 0:
        order = order[:k]
    w = np.exp((x[order] - x[order[0]]) / t)
    stay = np.ones(order.size, dtype=bool)
    if p is not None and p < 1:
        upto = np.cumsum(w)
        stay[1:] &= upto[:-1] < p * upto[-1]
    if m is not None:
        stay &= w >= min(m, 1.0)
    ids, w = order[stay], w[stay]
    by = np.argsort(ids)
    return ids[by], w[by]


def _rows(s):
    """(b, i, logits, temperature, top_k, top_p, min_p) of every position."""
    c = s["c"]
    t, k, p, m = _host(s, "temperature", "top_k", "top_p", "min_p")
    one = lambda a, b, f: None if a is None else f(a[b])  # noqa: E731
    for b in range(c["B"]):
        x = s["logits"][b].double().cpu().numpy()
        for i in range(c["P"]):
            yield b, i, x[i], float(t[b]), one(k, b, int), one(p, b, float), one(m, b, float)


def _exact_sample(s):
    c = s["c"]
    if c["B"] * c["P"] * c["V"] > 60_000_000:
        return None
    u = s["uniforms"].cpu().numpy().astype(np.float64)
    tokens = np.zeros((c["B"], c["P"], c["n"]), dtype=np.int32)
    logprobs = np.zeros((c["B"], c["P"], c["n"]))
    for b, i, x, t, k, p, m in _rows(s):
        if not t > 0:
            tokens[b, i] = np.argmax(x)
            continue
        ids, w = _kept_ids(x, t, k, p, m)
        upto = np.cumsum(w)
        for d in range(c["n"]):
            at = min(int(np.searchsorted(upto, u[b, i, d] * upto[-1], side="right")), ids.size - 1)
            tokens[b, i, d], logprobs[b, i, d] = ids[at], math.log(w[at] / upto[-1])
    return dict(tokens=tokens, logprobs=logprobs)


def _exact_truncate(s):
    c = s["c"]
    if c["B"] * c["P"] * c["V"] > 60_000_000:
        return None
    out = torch.full((c["B"], c["P"], c["V"]), -math.inf, dtype=torch.float64, device=DEV)
    for b, i, x, t, k, p, m in _rows(s):
        ids = torch.from_numpy(_kept_ids(x, t, k, p, m)[0] if t > 0 else np.arange(x.size)).to(DEV)
        out[b, i, ids] = s["logits"][b, i, ids].double()
    return out


def _path_of(par, v):
    """Nodes from the root to v."""
    path = [v]
    while path[-1] != 0:
        path.append(int(par[path[-1]]))
    return path[::-1]


def _exact_turn(x, s, ids):
    """Each pair as a complex number times e^(i angle)."""
    R = s["c"]["R"]
    x = x.double()
    if not R:
        return x
    first = torch.arange(0, R, 2, device=DEV) if s["c"]["interleaved"] else torch.arange(R // 2, device=DEV)
    second = first + (1 if s["c"]["interleaved"] else R // 2)
    angle = torch.empty(ids.shape[1:] + (R // 2,), dtype=torch.float64, device=DEV)
    for i in range(R // 2):
        angle[..., i] = ids[0 if s["axes"] is None else int(s["axes"][i])].double() * float(s["freqs"][i])
    z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(angle), angle)[:, :, None]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rotate(s):
    c = s["c"]
    ids = s["ids"]
    pos, par, lens = _host(s, "positions", "parents", "query_lens")
    if ids is None:
        at = np.zeros((1, c["B"], c["T"]))
        for b in range(c["B"]):
            at[0, b] = [pos[b] + (t if par is None else len(_path_of(par[b], t)) - 1) for t in range(c["T"])]
        ids = torch.from_numpy(at).to(DEV)
    q, k = _exact_turn(s["q"], s, ids), _exact_turn(s["k"], s, ids)
    if lens is not None:
        for b in range(c["B"]):
            q[b, lens[b]:] = 0
            k[b, lens[b]:] = 0
    return q, k


def _exact_append(s):
    c = s["c"]
    T, page = c["T"], c["page"]
    table, pos, blocks, lens = _host(s, "table", "positions", "blocks", "lens")
    R = s["k_tail"].shape[1]
    ids = s["ids"]
    if ids is None:
        ids = torch.from_numpy(pos[None, :, None] + np.arange(T)[None, None]).to(DEV)
    new = dict(k=_exact_turn(s["k"], s, ids), v=s["v"].double())
    # a key is a bf16 number before it is quantised; where 64 bits say which of two, it is that one
    new["k"] = new["k"].to(F32).to(BF16).double()
    kp, vp, ks, vs, kt, vt = (s[k].double() if k[2] != "p" else torch.zeros(s[k].shape, dtype=torch.float64, device=DEV)
                              for k in ("k_pages", "v_pages", "k_scale", "v_scale", "k_tail", "v_tail"))
    pos2, blocks2 = pos.copy(), blocks.copy()
    for b in range(c["B"]):
        n, tail = int(lens[b]), int(pos[b]) % page
        start, filled = int(pos[b]) - tail, (tail + n) // page
        pos2[b], blocks2[b] = pos[b] + n, blocks[b] + filled
        for x, pages, scales, ring in (("k", kp, ks, kt), ("v", vp, vs, vt)):
            slots = [(start + j) % R for j in range(tail)]
            seq = torch.cat([s[x + "_tail"][b, slots].double(), new[x][b, :n]])
            if filled:
                blk = seq[:filled * page].view(filled, page, c["Hkv"], c["D"]).transpose(1, 2)
                top = blk.abs().amax((2, 3))
                if c["kind"] == "int8":
                    scale = torch.where(top > 0, (top / 127).to(F32).double().clamp(min=2.0 ** -126), 1.0)
                    y = torch.round(blk / scale[..., None, None]) * scale[..., None, None]
                else:
                    scale = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)).clamp(min=-126))
                    scale = torch.where(top > 448 * scale, 2 * scale, scale)
                    scale = torch.where(top > 0, scale, 1.0)
                    y = blk / scale[..., None, None]
                    # steps of an eighth of the value's power of two, 2^-9 at least
                    step = torch.exp2((torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -20))) - 3).clamp(min=-9))
                    y = torch.round(y / step) * step
                at = torch.from_numpy(table[b, blocks[b]:blocks[b] + filled].astype(np.int64)).to(DEV)
                pages[at] = y if x == "k" else y.transpose(2, 3)
                scales[at] = scale
            for j in range(max(tail, filled * page), tail + n):
                ring[b, (start + j) % R] = seq[j]
    out = dict(k_pages=kp, v_pages=vp, k_scale=ks, v_scale=vs, k_tail=kt, v_tail=vt, positions=pos2, blocks=blocks2)
    if c["keys"]:
        out["k_out"] = new["k"].clone()
        for b in range(c["B"]):
            out["k_out"][b, lens[b]:] = 0
    return out


def _exact_prefix(s):
    c = s["c"]
    B, T, H, Hkv, D, page = (c[k] for k in ("B", "T", "H", "Hkv", "D", "page"))
    if sum(_queries(c)) * H * (c["prefix"] + c["ctx"]) * D > 3e10:
        return None
    table, shared, many, pos, blocks, par, nq = _host(s, "table", "prefix_table", "prefix_blocks", "positions",
                                                      "blocks", "parents", "query_lens")
    R = s["k_tail"].shape[1]
    out = torch.zeros((B, T, H, D), dtype=torch.float64, device=DEV)
    weights = torch.zeros((B, T, table.shape[1]), dtype=torch.float64, device=DEV)
    kind = torch.int8 if c["kind"] == "int8" else torch.float8_e4m3fn
    for b in range(B):
        n, tail = int(blocks[b]), int(pos[b]) % page
        t = T if nq is None else int(nq[b])
        first = shared[s["of"][b], :many[s["of"][b]]] if s["of"][b] >= 0 else shared[0, :0]
        before = len(first) * page
        near = before + n * page + tail
        see = torch.zeros((t, near + t), dtype=torch.bool)
        see[:, :near] = True
        for i in range(t):
            see[i, [near + j for j in (range(i + 1) if par is None else _path_of(par[b], i))]] = True
        see = see.to(DEV)
        pages = torch.from_numpy(np.concatenate([first, table[b, :n]]).astype(np.int64)).to(DEV)
        slots = torch.tensor([(int(pos[b]) - tail + j) % R for j in range(tail)], dtype=torch.long, device=DEV)
        for h in range(Hkv):
            k = s["k_pages"][pages, h].view(kind).to(torch.float64) * s["k_scale"][pages, h].double()[:, None, None]
            v = s["v_pages"][pages, h].view(kind).to(torch.float64) * s["v_scale"][pages, h].double()[:, None, None]
            k = torch.cat([k.reshape(-1, D), s["k_tail"][b, slots, h].double(), s["k_new"][b, :t, h].double()])
            v = torch.cat([v.transpose(1, 2).reshape(-1, D), s["v_tail"][b, slots, h].double(),
                           s["v_new"][b, :t, h].double()])
            for hq in range(h * (H // Hkv), (h + 1) * (H // Hkv)):
                z = torch.where(see, s["q"][b, :t, hq].double() @ k.T / math.sqrt(D), -math.inf)
                p = torch.softmax(z, 1)
                out[b, :t, hq] = p @ v
                weights[b, :t, :n] += p[:, before:before + n * page].reshape(t, n, page).sum(2)
    return (out, weights) if c["weights"] else out
