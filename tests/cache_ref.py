"""Random states of the paged 8-bit cache, and float64 references of the calls
that read and write it, in plain loops over rows and heads on the CPU."""

from __future__ import annotations

import numpy as np
import torch

import rejection_sampling_verifier_amd as rsv

BF16 = torch.bfloat16
NAN_CODE = 0x7F  # e4m3's NaN


def decode(codes, kind):
    """uint8 codes -> float64, by torch's own types."""
    if kind == "int8":
        return codes.view(torch.int8).to(torch.float64)
    return codes.view(torch.float8_e4m3fn).to(torch.float32).to(torch.float64)


def random_state(seed, *, B, Hkv, D, page, kind, contexts, evicted=None, max_blocks=None, max_new=65, spare=3,
                 bad_entries=()):
    """A cache (CPU tensors) whose rows hold `contexts` tokens (blocks kept, tail), the rest NaN.

    evicted: blocks each row lost before, so that positions run ahead.  bad_entries: (row, block, page id) to put in
    the table.  Unused pages, tail slots and (as their code has one) e4m3 codes are NaN; unused scales too.
    """
    g = torch.Generator().manual_seed(seed)
    blocks = [c // page for c in contexts]
    evicted = evicted or [0] * B
    most = max_blocks or max(blocks) + 2
    pages = sum(blocks) + spare
    tail = -(-(page - 1 + max_new) // page) * page
    table = torch.full((B, most), -1, dtype=torch.int32)
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    at = 0
    for b in range(B):
        table[b, :blocks[b]] = perm[at:at + blocks[b]]
        at += blocks[b]
    used = torch.zeros(pages, dtype=torch.bool)
    used[perm[:at].long()] = True
    if kind == "int8":
        code = lambda s: torch.randint(-128, 128, s, generator=g, dtype=torch.int16).to(torch.int8).view(torch.uint8)  # noqa: E731
    else:
        def code(s):
            c = torch.randint(0, 256, s, generator=g, dtype=torch.int16).to(torch.uint8)
            return torch.where((c & 0x7F) == 0x7F, c ^ 1, c)
    # e4m3 codes drawn evenly reach 448; scales that make values of about 1
    unit = 1 / 64 if kind == "int8" else 1 / 64
    s = dict(kind=kind, page=page, D=D, Hkv=Hkv, B=B)
    s["k_pages"], s["v_pages"] = code((pages, Hkv, page, D)), code((pages, Hkv, D, page))
    for k in ("k_scale", "v_scale"):
        s[k] = unit * (0.2 + torch.rand((pages, Hkv), generator=g))
        s[k][~used] = float("nan")
    if kind == "e4m3":
        s["k_pages"][~used] = NAN_CODE
        s["v_pages"][~used] = NAN_CODE
    for b, j, p in bad_entries:
        table[b, j] = p
    s["table"] = table
    s["positions"] = torch.tensor([c + e * page for c, e in zip(contexts, evicted)], dtype=torch.int32)
    s["blocks"] = torch.tensor(blocks, dtype=torch.int32)
    for k in ("k_tail", "v_tail"):
        x = torch.full((B, tail, Hkv, D), float("nan"), dtype=BF16)
        for b in range(B):
            for slot in tail_slots(s, b, tail):
                x[b, slot] = torch.randn((Hkv, D), generator=g).to(BF16)
        s[k] = x
    s["tail"] = tail
    return s


def tail_slots(s, b, tail):
    """Ring slots of row b's tail tokens, in order."""
    pos, page = int(s["positions"][b]), s["page"]
    n = pos % page
    return [(pos - n + j) % tail for j in range(n)]


TENSORS = ("k_pages", "v_pages", "k_scale", "v_scale", "k_tail", "v_tail", "table")


def to_gpu(s):
    """A KVCache over copies of the state's tensors, with its counters."""
    t = {k: s[k].cuda() for k in TENSORS}
    cache = rsv.KVCache(*(t[k] for k in TENSORS), kind=s["kind"])
    return cache, s["positions"].cuda(), s["blocks"].cuda()


def path_of(par, v):
    """Nodes from the root (or from a node with a bad parent) to v."""
    out = [v]
    while v > 0:
        p = int(par[v])
        if not 0 <= p < v:
            break
        v = p
        out.append(v)
    return out[::-1]


def visible(par, T, t):
    return list(range(t + 1)) if par is None else path_of(par, t)


def attention(s, q, k_new, v_new, scale, parents=None, query_lens=None):
    """float64 results: out [B, T, H, D], weights [B, T, max_blocks], and what bounds the error:
    av = sum p |v| (as out) and smax [B, T, H], the largest sum of |scale q_d k_d| over the keys seen."""
    B, T, H, D = q.shape
    Hkv, page, G = s["Hkv"], s["page"], H // s["Hkv"]
    most = s["table"].shape[1]
    out, av = torch.zeros((B, T, H, D), dtype=torch.float64), torch.zeros((B, T, H, D), dtype=torch.float64)
    weights, smax = torch.zeros((B, T, most), dtype=torch.float64), torch.zeros((B, T, H), dtype=torch.float64)
    for b in range(B):
        nq = T if query_lens is None else min(max(int(query_lens[b]), 0), T)
        n = min(max(int(s["blocks"][b]), 0), most)
        tail = tail_slots(s, b, s["k_tail"].shape[1])
        pages = [int(p) for p in s["table"][b, :n]]
        there = [j for j in range(n) if 0 <= pages[j] < s["k_pages"].shape[0]]
        at = torch.tensor([pages[j] for j in there], dtype=torch.long)
        for h in range(Hkv):
            k = decode(s["k_pages"][at, h], s["kind"]) * s["k_scale"][at, h].double()[:, None, None]
            v = decode(s["v_pages"][at, h], s["kind"]) * s["v_scale"][at, h].double()[:, None, None]
            k = torch.cat([k.reshape(-1, D), s["k_tail"][b, tail, h].double()])
            v = torch.cat([v.transpose(1, 2).reshape(-1, D), s["v_tail"][b, tail, h].double()])
            nc = k.shape[0]
            for t in range(nq):
                see = visible(None if parents is None else parents[b], T, t)
                kk = torch.cat([k, k_new[b, see, h].double()])
                vv = torch.cat([v, v_new[b, see, h].double()])
                qq = q[b, t, h * G:(h + 1) * G].double()
                p = torch.softmax(qq @ kk.T * scale, 1)
                out[b, t, h * G:(h + 1) * G] = p @ vv
                av[b, t, h * G:(h + 1) * G] = p @ vv.abs()
                smax[b, t, h * G:(h + 1) * G] = (qq.abs() @ kk.abs().T * scale).amax(1)
                mass = p[:, :len(there) * page].reshape(G, len(there), page).sum((0, 2))
                weights[b, t, there] += mass
                assert nc == len(there) * page + len(tail)
    return out, weights, av, smax


def as_numpy(t):
    return t.detach().cpu().double().numpy() if t.is_floating_point() else np.asarray(t.detach().cpu())


def scale_of(top, kind):
    """A block's scale for its largest magnitude (a float), as float64's value."""
    if not np.isfinite(top):
        return float("nan")
    if top == 0:
        return 1.0
    if kind == "int8":
        return max(float(np.float32(np.float64(top) / 127)), 2.0 ** -126)
    e = -126
    while top > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def quantise(x, kind):
    """x: float64 [page, D] -> (values the codes stand for / scale, scale); ties to even, by exact rationals."""
    top = float(x.abs().max()) if torch.isfinite(x).all() else float("inf")
    scale = scale_of(top, kind)
    if not np.isfinite(top):
        return torch.zeros_like(x), scale
    if kind == "int8":
        # bf16 / float32 in float64 is off by 2^-53: no tie is missed or made up, as 2 x / scale is an odd
        # integer only where the division is exact, and near ones differ from it by 2^-32 at least
        return torch.round(x / scale), scale
    y = x / scale
    step = torch.exp2((torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -30))) - 3).clamp(min=-9))
    return torch.round(y / step) * step, scale


def commit(s, k_new, v_new, num_accepted, nodes=None, weights=None, totals=None):
    """The state after a commit (a new dict), with totals.  Pages as values / scale (float64) in k_values, v_values:
    those written; NaN for the others."""
    page, D, Hkv, B = s["page"], s["D"], s["Hkv"], s["B"]
    T, most, pages, R = k_new.shape[1], s["table"].shape[1], s["k_pages"].shape[0], s["k_tail"].shape[1]
    new = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in s.items()}
    vals = {x: torch.full((pages, Hkv, page, D), float("nan"), dtype=torch.float64) for x in "kv"}
    tot = None if totals is None else torch.zeros_like(totals, dtype=torch.float64)
    for b in range(B):
        pos, blocks, n = int(s["positions"][b]), int(s["blocks"][b]), int(num_accepted[b]) + 1
        ok = 1 <= n <= T and 0 <= pos <= 2 ** 31 - 1 - n and 0 <= blocks <= most
        path = []
        if ok:
            path = [0] + [int(nodes[b, i]) if nodes is not None else i + 1 for i in range(n - 1)]
            ok = all(0 <= c < T for c in path)
            tail = pos % page
            filled = (tail + n) // page
            for m in range(filled):
                j = blocks + m
                ok = ok and j < most and 0 <= int(s["table"][b, j]) < pages
        if not ok:
            path, filled, n = [], 0, 0
        if tot is not None:
            keep = min(max(blocks, 0), most) if ok or 0 <= blocks <= most else (0 if blocks < 0 else most)
            tot[b, :keep] = totals[b, :keep].double()
            if weights is not None and path:
                tot[b, :keep] += weights[b, path, :keep].double().sum(0)
        if not ok:
            continue
        start = pos - tail
        for x, fresh in (("k", k_new), ("v", v_new)):
            seq = torch.cat([s[x + "_tail"][b, [(start + j) % R for j in range(tail)]].reshape(tail, Hkv, D),
                             fresh[b, path]])
            for m in range(filled):
                pid = int(s["table"][b, blocks + m])
                for h in range(Hkv):
                    y, scale = quantise(seq[m * page:(m + 1) * page, h].double(), s["kind"])
                    vals[x][pid, h] = y
                    new[x + "_scale"][pid, h] = scale
            for j in range(max(tail, filled * page), tail + n):
                new[x + "_tail"][b, (start + j) % R] = seq[j]
        new["positions"][b], new["blocks"][b] = pos + n, blocks + filled
    return new, vals, tot


def evict(table, totals, blocks, budget, first=0, last=0):
    table, totals, blocks = (t.clone().numpy() for t in (table, totals, blocks))
    gone = np.zeros_like(blocks)
    for b in range(table.shape[0]):
        n = min(max(int(blocks[b]), 0), table.shape[1])
        may = [j for j in range(n) if first <= j < n - last]
        e = min(max(0, n - budget), len(may))
        order = sorted(may, key=lambda j: ((1, 0.0) if np.isnan(totals[b, j]) else (0, float(totals[b, j])), j))
        away = set(order[:e])
        keep = [j for j in range(n) if j not in away]
        table[b, :n] = table[b, keep + sorted(away)]
        totals[b, :n - e] = totals[b, keep]
        totals[b, n - e:] = 0
        blocks[b], gone[b] = n - e, e
    return table, totals, blocks, gone
