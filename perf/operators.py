"""Workloads of the serving operators around the decode step: appending rotated
keys and values to a paged cache, attention of one new token over that cache,
causal attention over packed prompts, and sampling the next token.

Each case is one call as a serving loop makes it, with the head counts of the
shapes in workloads.py (tiny, 1B, 8B) or generic ones.  `run` is one pass:
the framework's call where `own` is true, else the same operator in plain
torch operations (32-bit arithmetic, 64-bit where angles, sums or borders
need it).  `exact` restates each operator in 64 bits, sequence by sequence.

Formulas.  d = head size, G = query heads per KV head, a sequence's rows are
consecutive tokens.
  append:  inv_i = theta^(-2i/d), a = position * inv_i, for i < d/2:
           x'_i = x_i cos a - x_{i+d/2} sin a,  x'_{i+d/2} = x_{i+d/2} cos a + x_i sin a
           for q and k; k' and v go to page table[seq][pos / page], row pos % page.
  paged:   o = sum_j softmax_j(q.k_j * scale) v_j over j < len (zero if len = 0).
  prompt:  the same for every token over the tokens of its sequence up to itself.
  sample:  w_i = exp((l_i - max l) / T); keep the top_k largest (ties: lowest
           index), of those the shortest descending prefix with top_p of their
           mass, of those w_i >= min_p; the first kept index whose running sum
           of w (in index order) exceeds u times the kept sum.  T = 0: argmax.
"""
import math
import random

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _mk():
    from persistent_decode_megakernel_02_b200 import mk
    return mk


# ---- cases --------------------------------------------------------------------

def listed():
    b1 = dict(q_heads=32, kv_heads=8, head_dim=64, theta=5e5)     # the 1B shape's heads
    b8 = dict(q_heads=32, kv_heads=8, head_dim=128, theta=5e5)    # the 8B shape's heads
    return [
        # one decode step's new tokens of 16 sequences at staggered positions
        dict(name="append_decode_16", op="append", seqs=16, max_new=1, max_start=2048, page=16,
             dtype="bf16", seed=1, ragged=False, **b1),
        # several prompts of odd lengths appended together, an empty one among them
        dict(name="append_prompts_ragged", op="append", seqs=7, max_new=391, max_start=900, page=64,
             dtype="fp16", seed=2, ragged=True, **b8),
        # a long prompt's chunk far into a long context
        dict(name="append_chunk_8k_far", op="append", seqs=1, max_new=8192, max_start=114688, page=128,
             dtype="bf16", seed=3, ragged=False, **b8),
        # batch-1 decode late in the benchmark's generation (39-token prompt, 512 steps)
        dict(name="paged_1x551", op="paged", seqs=1, max_len=551, page=16, dtype="bf16", seed=4,
             ragged=False, empty=False, **b1),
        # the batched decode sweep: 16 sequences at positions up to 2048
        dict(name="paged_16x2048_ragged", op="paged", seqs=16, max_len=2048, page=16, dtype="bf16",
             seed=5, ragged=True, empty=False, **b1),
        # batch-1 decode over the long-context workload's cache
        dict(name="paged_1x16385", op="paged", seqs=1, max_len=16385, page=64, dtype="bf16", seed=6,
             ragged=False, empty=False, **b1),
        # a serving batch of long and short sequences, one slot idle
        dict(name="paged_32x16384_ragged", op="paged", seqs=32, max_len=16384, page=128, dtype="fp16",
             seed=7, ragged=True, empty=True, **b8),
        # the benchmark's prompt
        dict(name="prompt_39", op="prompt", seqs=1, max_len=39, dtype="bf16", seed=8, ragged=False,
             empty=False, **b1),
        # prompts of different lengths packed into one call
        dict(name="prompt_9_packed", op="prompt", seqs=9, max_len=1511, dtype="fp16", seed=9, ragged=True,
             empty=True, **b1),
        # a long document
        dict(name="prompt_8192", op="prompt", seqs=1, max_len=8192, dtype="bf16", seed=10, ragged=False,
             empty=False, **b8),
        # batch-1 decode: one row of the models' vocabulary, every filter on
        dict(name="sample_1_filtered", op="sample", rows=1, vocab=128256, mode="filtered", ties=False),
        # a serving batch whose requests ask for different things, logits from a 16-bit head
        dict(name="sample_64_mixed", op="sample", rows=64, vocab=128256, mode="mixed", ties=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "paged", "prompt", "sample"])
    if op == "sample":
        return dict(op=op, rows=_log_int(rng, 1, 64), vocab=_log_int(rng, 1000, 128256),
                    mode=rng.choice(["plain", "filtered", "mixed"]), ties=rng.random() < 0.3)
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 6, 8])
    group = group if kv * group <= 32 else 4
    heads = dict(q_heads=kv * group, kv_heads=kv, head_dim=rng.choice([64, 128]), theta=rng.choice([1e4, 5e5]),
                 dtype=rng.choice(["bf16", "fp16"]), seed=rng.randrange(1 << 30))
    page = rng.choice([16, 32, 64, 128, 24, 50, 560])
    if op == "append":
        seqs = _log_int(rng, 1, 64)
        new = 1 if rng.random() < 0.4 else _log_int(rng, 1, 8192 // seqs)
        return dict(op=op, seqs=seqs, max_new=new, max_start=_log_int(rng, 1, 120000), page=page,
                    ragged=new > 1 and rng.random() < 0.7, **heads)
    if op == "paged":
        seqs = _log_int(rng, 1, 64)
        return dict(op=op, seqs=seqs, max_len=_log_int(rng, 1, 262144 // max(seqs, 4)), page=page,
                    ragged=rng.random() < 0.7, empty=seqs > 1 and rng.random() < 0.3, **heads)
    seqs = _log_int(rng, 1, 16)
    return dict(op=op, seqs=seqs, max_len=_log_int(rng, 1, 8000 // seqs), ragged=rng.random() < 0.7,
                empty=seqs > 1 and rng.random() < 0.3, **heads)


def _lengths(case):
    """Per-sequence lengths (append: of the new tokens) and start positions."""
    rng = random.Random(case["seed"])
    n, top = case["seqs"], case["max_new"] if case["op"] == "append" else case["max_len"]
    lens = [rng.randint(1, top) if case["ragged"] else top for _ in range(n)]
    if case["ragged"]:
        lens[-1] = top
    if n > 1 and (case.get("empty") or case["op"] == "append" and case["ragged"]):
        lens[n // 2] = 0
    starts = [0] * n
    if case["op"] == "append":
        starts = [rng.randint(0, case["max_start"]) for _ in range(n)]
        if n == 1:
            starts = [case["max_start"]]
    return lens, starts


def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": 4 * n + 24 * case["rows"], "flops": 4 * n}
    lens, _ = _lengths(case)
    nq, nkv, d, t = case["q_heads"], case["kv_heads"], case["head_dim"], sum(lens)
    if case["op"] == "append":
        # q in and out; k in, out and into the cache; v in and into the cache
        return {"bytes": t * d * 2 * (2 * nq + 3 * nkv + 2 * nkv), "flops": 3 * t * d * (nq + nkv)}
    if case["op"] == "paged":
        return {"bytes": 2 * t * nkv * d * 2 + 2 * len(lens) * nq * d * 2, "flops": 4 * t * nq * d}
    return {"bytes": t * d * 2 * (2 * nq + 2 * nkv), "flops": sum(2 * n * (n + 1) for n in lens) * nq * d}


# ---- inputs --------------------------------------------------------------------

def _ints(values, device="cuda"):
    return torch.tensor(values, dtype=torch.int32).to(device)


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "sample":
        return _prepare_sample(case, g, seed)
    dt = _DTYPES[case["dtype"]]
    nq, nkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    lens, starts = _lengths(case)
    total, cu = sum(lens), _cu(lens)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    s = {"case": case, "op": case["op"]}
    if case["op"] == "prompt":
        s.update(q=randn(total, nq, d), k=randn(total, nkv, d), v=randn(total, nkv, d), cu=_ints(cu),
                 max_len=max(lens), out=torch.empty(total, nq, d, device="cuda", dtype=dt))
        return s
    # a pool of pages handed out in no order; the table's entries beyond a
    # sequence's own pages name some valid page
    page = case["page"]
    first = [a // page for a in starts]
    last = [(a + n + page - 1) // page for a, n in zip(starts, lens)]
    used = sum(b - a for a, b in zip(first, last) if b > a)
    perm = np.random.default_rng(seed).permutation(used + 1).astype(np.int32)
    table, at = np.full((len(lens), max(max(last), 1)), perm[used], np.int32), 0
    for i, (a, b) in enumerate(zip(first, last)):
        if b > a:
            table[i, a:b] = perm[at:at + b - a]
            at += b - a
    k_pages, v_pages = randn(used + 1, nkv, page, d), randn(used + 1, nkv, page, d)
    s.update(k_pages=k_pages, v_pages=v_pages, table=torch.from_numpy(table).cuda())
    if own:
        s["cache"] = _mk().PagedKV(k_pages, v_pages, s["table"])
    if case["op"] == "append":
        s.update(q=randn(total, nq, d), k=randn(total, nkv, d), v=randn(total, nkv, d), cu=_ints(cu),
                 start=_ints(starts), theta=case["theta"], q_out=torch.empty(total, nq, d, device="cuda", dtype=dt),
                 k_out=torch.empty(total, nkv, d, device="cuda", dtype=dt))
    else:
        s.update(q=randn(len(lens), nq, d), lens=_ints(lens), max_len=max(lens),
                 out=torch.empty(len(lens), nq, d, device="cuda", dtype=dt))
        if own:
            s["workspace"] = _mk().paged_attention_workspace(s["cache"], nq, s["max_len"])
    return s


def _prepare_sample(case, g, seed):
    rows, vocab, rng = case["rows"], case["vocab"], random.Random(seed)
    # a broad bulk and a few dozen plausible tokens above it, sharper in some rows than in others
    spread = torch.tensor([rng.uniform(1.0, 3.0) for _ in range(rows)], device="cuda")
    logits = torch.randn(rows, vocab, generator=g, device="cuda") * spread[:, None]
    at = torch.randint(0, vocab, (rows, 40), generator=g, device="cuda")
    logits.scatter_add_(1, at, 2.5 * spread[:, None] * torch.rand(rows, 40, generator=g, device="cuda"))
    if case["ties"]:
        logits = logits.bfloat16().float()
    params = []
    for _ in range(rows):
        t, k, p, m = rng.uniform(0.6, 1.3), rng.choice([20, 40, 50, 200]), rng.uniform(0.8, 0.98), rng.uniform(0.01, 0.1)
        if case["mode"] == "plain":
            k, p, m = 0, 1.0, 0.0
        elif case["mode"] == "mixed":
            which = rng.randrange(6)
            t = 0.0 if which == 0 else t
            k = k if which in (1, 4) else 0
            p = p if which in (2, 4) else 1.0
            m = m if which in (3, 4) else 0.0
        params.append((t, k, p, m))
    t, k, p, m = zip(*params)

    def floats(v):
        return torch.tensor(v, dtype=torch.float32).cuda()

    return {"op": "sample", "logits": logits, "temperature": floats(t), "top_k": _ints(k), "top_p": floats(p),
            "min_p": floats(m), "uniform": torch.rand(rows, generator=g, device="cuda"),
            "token": torch.empty(rows, dtype=torch.int32, device="cuda")}


# ---- one pass --------------------------------------------------------------------

def run(s):
    if own:
        mk = _mk()
        if s["op"] == "append":
            mk.kv_append(s["cache"], s["q"], s["k"], s["v"], s["cu"], s["start"], s["theta"], s["q_out"], s["k_out"])
            return s["q_out"], s["k_out"], s["k_pages"], s["v_pages"]
        if s["op"] == "paged":
            mk.paged_attention(s["cache"], s["q"], s["lens"], s["max_len"], s["out"], s["workspace"])
            return s["out"]
        if s["op"] == "prompt":
            mk.prompt_attention(s["q"], s["k"], s["v"], s["cu"], s["max_len"], s["out"])
            return s["out"]
        mk.sample(s["logits"], s["uniform"], s["token"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])
        return s["token"]
    return _PLAIN[s["op"]](s)


def _token_places(cu, total):
    """Sequence of each packed token, and its place within the sequence."""
    tok = torch.arange(total, device=cu.device)
    seq = torch.searchsorted(cu.long(), tok, right=True) - 1
    return seq, tok - cu.long()[seq]


def _plain_append(s):
    q, k, v, table, page = s["q"], s["k"], s["v"], s["table"], s["k_pages"].shape[2]
    d = q.shape[2]
    seq, place = _token_places(s["cu"], q.shape[0])
    pos = s["start"].long()[seq] + place
    inv = s["theta"] ** (-2.0 * torch.arange(d // 2, device=q.device, dtype=torch.float64) / d)
    angle = pos.double()[:, None] * inv
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def rotate(x):
        a, b = x.float().chunk(2, dim=-1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1).to(x.dtype)

    q_rot, k_rot = rotate(q), rotate(k)
    at, row = table[seq, pos // page].long(), pos % page
    s["k_pages"][at, :, row] = k_rot
    s["v_pages"][at, :, row] = v
    return q_rot, k_rot, s["k_pages"], s["v_pages"]


def _softmax_rows(scores):
    """exp(s - max s) and its sum; rows with nothing left give zeros and a one."""
    top = scores.amax(dim=-1, keepdim=True)
    e = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(dim=-1, keepdim=True)
    return e, torch.where(total == 0, torch.ones_like(total), total)


def _plain_paged(s):
    q, table = s["q"], s["table"].long()
    n, nq, d = q.shape
    nkv, page = s["k_pages"].shape[1:3]
    table = table[:, :(s["max_len"] + page - 1) // page]

    def gather(pages):   # [n][kv heads][positions][d]
        return pages[table].transpose(1, 2).reshape(n, nkv, -1, d).float()

    k, v = gather(s["k_pages"]), gather(s["v_pages"])
    beyond = torch.arange(k.shape[2], device=q.device) >= s["lens"][:, None]
    v = v.masked_fill(beyond[:, None, :, None], 0.0)
    scores = q.float().reshape(n, nkv, nq // nkv, d) @ k.transpose(2, 3) * d ** -0.5
    e, total = _softmax_rows(scores.masked_fill(beyond[:, None, None], -math.inf))
    return (e @ v / total).reshape(n, nq, d).to(q.dtype)


def _plain_prompt(s):
    q, k, v, cu, top = s["q"], s["k"], s["v"], s["cu"].long(), s["max_len"]
    total, nq, d = q.shape
    nkv = k.shape[1]
    n = cu.shape[0] - 1
    place = torch.arange(top, device=q.device)
    at = (cu[:-1, None] + place).clamp(max=max(total - 1, 0))

    def padded(x):       # [n][heads][positions][d]
        return x[at].transpose(1, 2).float()

    qp = padded(q).reshape(n, nkv, nq // nkv, top, d)
    scores = qp @ padded(k)[:, :, None].transpose(3, 4)
    scores *= d ** -0.5
    lens = (cu[1:] - cu[:-1])[:, None]
    seen = (place[None, :] <= place[:, None])[None] & (place < lens)[:, None]     # [n][queries][keys]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    vp = padded(v).masked_fill((place >= lens)[:, None, :, None], 0.0)
    e, norm = _softmax_rows(scores)
    out = (e @ vp[:, :, None] / norm).reshape(n, nq, top, d)
    seq, row = _token_places(s["cu"], total)
    return out[seq, :, row].to(q.dtype)


def _plain_sample(s):
    logits = s["logits"].double()
    vocab = logits.shape[1]
    t = s["temperature"].double()[:, None]
    greedy = t <= 0
    value, index = torch.sort(logits, dim=1, descending=True, stable=True)
    w = torch.exp((value - value[:, :1]) / torch.where(greedy, torch.ones_like(t), t))
    k = s["top_k"].long()[:, None]
    k = torch.where((k <= 0) | (k > vocab), torch.full_like(k, vocab), k)
    kept = w * (torch.arange(vocab, device=w.device) < k)
    before = kept.cumsum(dim=1) - kept
    p = s["top_p"].double()[:, None]
    in_p = (before < p * kept.sum(dim=1, keepdim=True)) | (p >= 1)
    in_p[:, 0] = True
    kept = kept * in_p * (w >= s["min_p"].double()[:, None])
    kept = torch.zeros_like(kept).scatter_(1, index, kept)      # back in index order
    run_sum = kept.cumsum(dim=1)
    target = s["uniform"].double()[:, None] * run_sum[:, -1:]
    token = torch.searchsorted(run_sum, target, right=True).clamp(max=vocab - 1)
    return torch.where(greedy, index[:, :1], token)[:, 0].int()


_PLAIN = {"append": _plain_append, "paged": _plain_paged, "prompt": _plain_prompt, "sample": _plain_sample}


# ---- the definitions in 64 bits ----------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(s)
    lens, starts = _lengths(case)
    cu = _cu(lens)
    d, group = case["head_dim"], case["q_heads"] // case["kv_heads"]
    if case["op"] == "append":
        pos = torch.tensor([a + i for a, n in zip(starts, lens) for i in range(n)], dtype=torch.float64, device="cuda")
        # half-split pairs as complex numbers, turned by the angle
        turn = torch.exp(1j * torch.outer(pos, torch.exp(-math.log(case["theta"]) * 2.0 / d *
                                                         torch.arange(d // 2, dtype=torch.float64, device="cuda"))))

        def rotate(x):
            z = torch.complex(x[..., :d // 2].double(), x[..., d // 2:].double()) * turn[:, None]
            return torch.cat([z.real, z.imag], dim=-1)

        q, k = rotate(s["q"]), rotate(s["k"])
        kp, vp, table, page = s["k_pages"].double(), s["v_pages"].double(), s["table"].tolist(), case["page"]
        for b, n in enumerate(lens):
            i = 0
            while i < n:        # the rows of one page at a time
                p, r = divmod(starts[b] + i, page)
                m = min(n - i, page - r)
                kp[table[b][p], :, r:r + m] = k[cu[b] + i:cu[b] + i + m].transpose(0, 1)
                vp[table[b][p], :, r:r + m] = s["v"][cu[b] + i:cu[b] + i + m].transpose(0, 1).double()
                i += m
        return q, k, kp, vp
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n == 0:
            continue
        for h in range(case["kv_heads"]):
            heads = slice(h * group, (h + 1) * group)
            if case["op"] == "paged":
                page = case["page"]
                pages = s["table"][b, :(n + page - 1) // page].long()
                k = s["k_pages"][pages, h].reshape(-1, d)[:n].double()
                v = s["v_pages"][pages, h].reshape(-1, d)[:n].double()
                out[b, heads] = torch.softmax(s["q"][b, heads].double() @ k.T / math.sqrt(d), dim=-1) @ v
                continue
            rows = slice(cu[b], cu[b + 1])
            k, v = s["k"][rows, h].double(), s["v"][rows, h].double()
            later = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
            for hq in range(h * group, (h + 1) * group):
                sc = s["q"][rows, hq].double() @ k.T / math.sqrt(d)
                out[rows, hq] = torch.softmax(sc.masked_fill_(later, -math.inf), dim=-1) @ v
    return out


def _exact_sample(s):
    logits = s["logits"].double().cpu().numpy()
    par = [s[n].cpu().numpy() for n in ("temperature", "top_k", "top_p", "min_p", "uniform")]
    tokens = []
    for row, t, k, p, m, u in zip(logits, *par):
        if t <= 0:
            tokens.append(int(np.argmax(row)))
            continue
        w = np.exp((row - row.max()) / float(t))
        order = np.argsort(-row, kind="stable")
        if 0 < k < len(row):
            order = order[:k]
        if p < 1:
            mass = np.cumsum(w[order])
            order = order[:int(np.searchsorted(mass, float(p) * mass[-1], side="left")) + 1]
        keep = np.zeros(len(row), bool)
        keep[order] = True
        keep &= w >= float(m)
        at = np.flatnonzero(keep)
        run_sum = np.cumsum(w[at])
        tokens.append(int(at[min(int(np.searchsorted(run_sum, float(u) * run_sum[-1], side="right")), len(at) - 1)]))
    return torch.tensor(tokens, dtype=torch.int32)
