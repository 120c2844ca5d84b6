"""Speed of the serving operators over a paged K/V cache, and of the prompt's attention weights.

Each case is one pass through one operator, as a serving program calls it:

* ``tree``     attention of a tree of drafted tokens over a paged cache (decode_tree_paged);
* ``sparse``   one decode step that picks the best cache blocks of each KV head by the bound that
               the blocks' key ranges put on their scores, and attends to those (select_blocks,
               decode_paged_selected);
* ``bounds``   the blocks' key ranges that the choice reads (block_key_bounds);
* ``weights``  a decode step that also adds up the attention weight of every cached key
               (decode_paged_weights);
* ``prompt``   the attention weight that a prompt's queries put on its keys
               (attention_packed_weights);
* ``evict``    the keys with the least weight leave the cache (evict_paged).

``own`` false: the operators in plain torch operations. ``own`` true: the framework's calls.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    """Twelve cases: for each operator a call where latency counts and one of full size."""
    return [
        # One user, eight drafted tokens, the heads of the packed example.
        {"name": "tree_1x8_ctx777", "op": "tree", "n": 1, "lo": 777, "hi": 777, "ls": 1, "hq": 8,
         "hkv": 8, "d": 64, "dtype": "fp16", "bs": 16, "draft": 8, "alibi": False},
        # A batch of verification steps over the decode workload's lengths and heads.
        {"name": "tree_16x32_ctx32k", "op": "tree", "n": 16, "lo": 512, "hi": 32768, "ls": 2,
         "hq": 64, "hkv": 8, "d": 128, "dtype": "bf16", "bs": 64, "draft": 32, "alibi": False},
        # One long chat, 16-slot blocks, 1024 of 20001 keys.
        {"name": "sparse_1x20001", "op": "sparse", "n": 1, "lo": 20001, "hi": 20001, "ls": 3,
         "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16", "bs": 16, "select": 64, "alibi": False},
        # The decode workload, 2048 keys a head.
        {"name": "sparse_64x32k", "op": "sparse", "n": 64, "lo": 512, "hi": 32768, "ls": 4,
         "hq": 64, "hkv": 8, "d": 128, "dtype": "bf16", "bs": 32, "select": 64, "alibi": False},
        # After a decode step: only the block of the newest key changed.
        {"name": "bounds_step_64", "op": "bounds", "n": 64, "lo": 512, "hi": 8192, "ls": 5,
         "hq": 64, "hkv": 8, "d": 128, "dtype": "bf16", "bs": 16, "newest": 1},
        # After the prompts were written: every block.
        {"name": "bounds_prompts_16", "op": "bounds", "n": 16, "lo": 512, "hi": 32768, "ls": 6,
         "hq": 64, "hkv": 8, "d": 128, "dtype": "bf16", "bs": 32, "newest": 0},
        # A small model's single user.
        {"name": "weights_1x3001", "op": "weights", "n": 1, "lo": 3001, "hi": 3001, "ls": 7,
         "hq": 8, "hkv": 8, "d": 64, "dtype": "fp16", "bs": 16, "prev": True, "alibi": True},
        # The decode workload, weights added up over the steps.
        {"name": "weights_64x32k", "op": "weights", "n": 64, "lo": 512, "hi": 32768, "ls": 8,
         "hq": 64, "hkv": 8, "d": 128, "dtype": "bf16", "bs": 64, "prev": True, "alibi": False},
        # The weights that the last 32 queries of each prompt of the packed workload put on it.
        {"name": "prompt_packed_last32", "op": "prompt", "n": 16, "lo": 64, "hi": 4096, "ls": 9,
         "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16", "last": 32, "alibi": True},
        # Every query of the long prefill.
        {"name": "prompt_16k_all", "op": "prompt", "n": 1, "lo": 16384, "hi": 16384, "ls": 10,
         "hq": 64, "hkv": 8, "d": 128, "dtype": "bf16", "last": 0, "alibi": False},
        # One chat outgrows its share of the cache.
        {"name": "evict_1x5003", "op": "evict", "n": 1, "lo": 5003, "hi": 5003, "ls": 11,
         "hq": 8, "hkv": 8, "d": 64, "dtype": "fp16", "bs": 16, "keep": 1024, "recent": 64},
        # A full batch is cut to 4096 keys a head.
        {"name": "evict_64x32k", "op": "evict", "n": 64, "lo": 512, "hi": 32768, "ls": 12,
         "hq": 64, "hkv": 8, "d": 128, "dtype": "bf16", "bs": 32, "keep": 4096, "recent": 256},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges; costs no more than the largest listed one of its kind."""
    while True:
        op = rng.choice(["tree", "sparse", "bounds", "weights", "prompt", "evict"])
        hq, hkv = rng.choice([(64, 8), (32, 8), (8, 8), (8, 2), (12, 4), (16, 1)])
        c = {"op": op, "n": _log_uniform(rng, 1, 64), "hq": hq, "hkv": hkv,
             "d": rng.choice([64, 128, 128, 80, 256 if op != "prompt" else 96]),
             "dtype": rng.choice(["bf16", "fp16"]), "ls": rng.randrange(1 << 30)}
        hi = _log_uniform(rng, 1, 32768 if op != "prompt" else 16384)
        c["hi"] = hi
        c["lo"] = rng.choice([hi, max(1, hi // 8), max(1, hi // 64)])
        if op != "prompt":
            c["bs"] = rng.choice([16, 32, 64, 128])
        if op == "tree":
            c["draft"] = min(_log_uniform(rng, 1, 64), c["lo"])
            c["alibi"] = rng.random() < 0.3
        elif op == "sparse":
            c["select"] = _log_uniform(rng, 1, 128)
            c["alibi"] = rng.random() < 0.3
        elif op == "bounds":
            c["newest"] = rng.choice([0, 1, _log_uniform(rng, 1, 4096)])
        elif op == "weights":
            c["prev"] = rng.random() < 0.7
            c["alibi"] = rng.random() < 0.3
        elif op == "prompt":
            c["last"] = rng.choice([0, _log_uniform(rng, 1, 256)])
            c["alibi"] = rng.random() < 0.3
        else:
            c["keep"] = _log_uniform(rng, 1, 4096)
            c["recent"] = rng.randrange(0, c["keep"] + 1)
        # the plain forms' padded reads, and the products, within the largest listed case's
        if c["n"] * c["hi"] * hkv * c["d"] > 64 * 32768 * 8 * 128:
            continue
        if op == "tree" and c["n"] * c["hi"] * c["draft"] * hq * c["d"] > \
                16 * 32768 * 32 * 64 * 128:
            continue
        if op == "prompt" and (c["n"] * c["hi"] * c["hi"] * hq * c["d"] >
                               16384 * 16384 * 64 * 128 or
                               c["n"] * c["hi"] * (c["last"] or c["hi"]) > 16384 * 16384):
            continue
        return c


def _lens(case):
    """The requests' key counts (a prompt's tokens), from the case alone."""
    r = random.Random(case["ls"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["n"])]


def _drafts(case):
    """The requests' drafted tokens: the full draft or up to half of it less."""
    r = random.Random(case["ls"] + 1)
    return [r.randint((case["draft"] + 1) // 2, case["draft"]) for _ in range(case["n"])]


def _cu(lens):
    c = [0]
    for x in lens:
        c.append(c[-1] + x)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def _slopes(hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], dtype=torch.float32,
                        device="cuda")


def prepare(case, seed):
    """What a serving program holds before the call."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, d, hq, hkv, n = DT[case["dtype"]], case["d"], case["hq"], case["hkv"], case["n"]
    lens = _lens(case)
    s = {"case": case, "lens": lens, "max": max(lens), "cu": _cu(lens), "scale": d ** -0.5,
         "len_t": torch.tensor(lens, device="cuda"),
         "slopes": _slopes(hq) if case.get("alibi") else None}

    def rand(*shape, dtype=dt):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    if case["op"] == "prompt":
        total = sum(lens)
        s["q"] = rand(total, hq, d)
        s["k"] = rand(total, hkv, d)
        # The log-sum-exps that the prompt's attention call left.
        lse = torch.empty((hq, total), dtype=torch.float32, device="cuda")
        off = 0
        for length in lens:
            i = torch.arange(length, device="cuda")
            for h in range(hq):
                x = s["q"][off:off + length, h].float() @ \
                    s["k"][off:off + length, h // (hq // hkv)].float().t()
                x *= s["scale"]
                if s["slopes"] is not None:
                    x -= s["slopes"][h] * (i[:, None] - i[None, :])
                x.masked_fill_(i[None, :] > i[:, None], -math.inf)
                lse[h, off:off + length] = torch.logsumexp(x, 1)
            off += length
        s["lse"] = lse
        s["weights"] = torch.zeros((n, hkv, s["max"]), dtype=torch.float32, device="cuda")
        s["pad"] = _padding(lens, s["max"])
        return s

    bs = case["bs"]
    nblk = [-(-x // bs) for x in lens]
    num_blocks = sum(nblk) + 3
    perm = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((n, max(nblk)), dtype=torch.int32, device="cuda")
    off = 0
    for b in range(n):
        table[b, :nblk[b]] = perm[off:off + nblk[b]]
        off += nblk[b]
    # Keys of one block share a part, as neighbouring tokens' keys do.
    k_cache = rand(num_blocks, bs, hkv, d)
    k_cache += 0.5 * rand(num_blocks, 1, hkv, d)
    s["k_cache"], s["table"], s["total"] = k_cache, table, sum(lens)
    # The cache row of each request's keys (rows of no key: row 0), for the plain forms.
    j = torch.arange(s["max"], device="cuda")
    s["valid"] = j[None, :] < s["len_t"][:, None]
    s["rows"] = (table.long()[:, j // bs] * bs + j % bs).masked_fill_(~s["valid"], 0)
    if case["op"] in ("tree", "sparse", "weights"):
        s["v_cache"] = rand(num_blocks, bs, hkv, d)
        s["q"] = rand(n, hq, d)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((hq, n), dtype=torch.float32, device="cuda")
    if case["op"] == "tree":
        drafts = _drafts(case)
        words = (max(drafts) + 31) // 32
        r, bits = random.Random(seed), []
        for x in drafts:
            seen = []
            for i in range(x):
                p = r.randint(-1, i - 1)
                seen.append((seen[p] if p >= 0 else 0) | (1 << i))
            bits += seen
        rows = [[((m >> (32 * w)) & 0xffffffff) for w in range(words)] for m in bits]
        s["mask"] = torch.tensor(rows, dtype=torch.int64, device="cuda").to(torch.int32)
        s["cu_q"], s["max_q"] = _cu(drafts), max(drafts)
        s["draft_t"] = torch.tensor(drafts, device="cuda")
        s["pad"] = _padding(drafts, max(drafts))
        s["q"] = rand(sum(drafts), hq, d)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((hq, sum(drafts)), dtype=torch.float32, device="cuda")
    elif case["op"] in ("sparse", "bounds"):
        bounds = torch.zeros((num_blocks, hkv, 2, d), dtype=dt, device="cuda")
        if case["op"] == "sparse":
            for b in range(n):
                ids = table[b, :nblk[b]].long()
                x = k_cache[ids]
                dead = torch.arange(nblk[b] * bs, device="cuda").view(-1, bs) >= lens[b]
                x = x.masked_fill(dead[:, :, None, None], math.inf)
                bounds[ids, :, 0] = x.amin(1)
                bounds[ids, :, 1] = x.masked_fill(dead[:, :, None, None], -math.inf).amax(1)
            s["selected"] = torch.empty((n, hkv, case["select"]), dtype=torch.int32,
                                        device="cuda")
        else:
            new = case["newest"]
            s["first"] = (s["len_t"] - new).clamp_min(0).to(torch.int32) if new else None
        s["bounds"] = bounds
    elif case["op"] == "weights":
        s["weights"] = torch.zeros((n, hkv, s["max"]), dtype=torch.float32, device="cuda")
        s["prev"] = rand(n, hkv, s["max"], dtype=torch.float32).abs() if case["prev"] else None
    elif case["op"] == "evict":
        s["v_cache"] = rand(num_blocks, bs, hkv, d)
        s["weights"] = torch.exp(2 * rand(n, hkv, s["max"], dtype=torch.float32))
        keep = case["keep"]
        per = -(-keep // bs)
        s["out_table"] = torch.randperm(n * per, generator=g, device="cuda").to(torch.int32) \
            .view(n, per).contiguous()
        s["out_k"] = torch.zeros((n * per, bs, hkv, d), dtype=dt, device="cuda")
        s["out_v"] = torch.zeros_like(s["out_k"])
        s["out_weights"] = torch.zeros((n, hkv, keep), dtype=torch.float32, device="cuda")
        s["kept"] = torch.empty((n, hkv, keep), dtype=torch.int32, device="cuda")
        s["out_cu"] = torch.empty(n + 1, dtype=torch.int32, device="cuda")
    return s


def _padding(lens, width):
    """Between packed rows and rows padded to `width` a sequence: (sequence, place) of each packed
    row, the packed row of each place (0 where there is none), and which places have one."""
    n, device = len(lens), "cuda"
    lt = torch.tensor(lens, device=device)
    at = torch.arange(width, device=device)
    valid = at[None, :] < lt[:, None]
    start = torch.cumsum(lt, 0) - lt
    row = (start[:, None] + at[None, :]).masked_fill(~valid, 0)
    seq = torch.repeat_interleave(torch.arange(n, device=device), lt)
    place = torch.arange(int(sum(lens)), device=device) - start[seq]
    return {"seq": seq, "place": place, "row": row, "valid": valid}


# ------------------------------------------------------------------------------------------
# Plain forms: elementary torch operations in 32 bits, all requests at once.
# ------------------------------------------------------------------------------------------
def _softmax(x):
    """Row softmax of masked scores (-inf: masked) and its log-sum-exp; an empty row gives 0, -inf."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    lse = torch.log(z) + m
    return e / torch.where(z > 0, z, torch.ones_like(z)), lse[..., 0]


def _gather(cache, rows):
    """Cache rows [n, keys] -> [n, hkv, keys, d] in 32 bits."""
    return cache.flatten(0, 1)[rows].permute(0, 2, 1, 3).float()


def _plain_decode(s, rows, keys, valid):
    """Single-token attention over gathered rows: rows/keys/valid [n, t] or, by KV head,
    [n, hkv, t]. Returns the weights [n, hkv, r, t], out and lse."""
    c = s["case"]
    n, hq, d = s["q"].shape
    hkv, r = c["hkv"], hq // c["hkv"]
    if rows.dim() == 2:
        k, v = _gather(s["k_cache"], rows), _gather(s["v_cache"], rows)
        keys, valid = keys[:, None], valid[:, None]
    else:
        head = torch.arange(hkv, device="cuda")[None, :, None]
        k = s["k_cache"].flatten(0, 1)[rows, head].float()
        v = s["v_cache"].flatten(0, 1)[rows, head].float()
    x = (s["q"].float().view(n, hkv, r, d) @ k.transpose(2, 3)) * s["scale"]
    if s["slopes"] is not None:
        dist = (s["len_t"][:, None, None] - 1 - keys).float()
        x = x - s["slopes"].view(1, hkv, r, 1) * dist[:, :, None, :]
    p, lse = _softmax(x.masked_fill(~valid[:, :, None, :], -math.inf))
    out = (p @ v).reshape(n, hq, d).to(s["q"].dtype)
    return p, out, lse.reshape(n, hq).t().contiguous()


def _plain_tree(s):
    c, pad = s["case"], s["pad"]
    hkv, d = c["hkv"], c["d"]
    r, n, w = c["hq"] // hkv, c["n"], s["max_q"]
    q = s["q"][pad["row"]].float().view(n, w, hkv, r, d).permute(0, 2, 1, 3, 4)
    k, v = _gather(s["k_cache"], s["rows"]), _gather(s["v_cache"], s["rows"])
    x = (q.reshape(n, hkv, w * r, d) @ k.transpose(2, 3)) * s["scale"]
    x = x.view(n, hkv, w, r, -1)
    t = torch.arange(s["max"], device="cuda")
    ctx = s["len_t"] - s["draft_t"]
    j = t[None, :] - ctx[:, None]  # draft index of each key, negative in the context
    bits = (s["mask"].long()[:, :, None] >> torch.arange(32, device="cuda")) & 1
    bits = bits.flatten(1).bool()[pad["row"]]  # [n, w, 32 * words]
    jc = j.clamp(0, bits.shape[2] - 1)
    seen = torch.gather(bits, 2, jc[:, None, :].expand(-1, w, -1)) | (j < 0)[:, None, :]
    seen = seen & s["valid"][:, None, :]
    if s["slopes"] is not None:
        depth = bits.sum(2) - 1  # ancestors of each drafted token, itself not counted
        dk = torch.gather(depth, 1, j.clamp(0, w - 1))
        kpos = torch.where(j < 0, t[None, :], ctx[:, None] + dk)
        dist = (ctx[:, None, None] + depth[:, :, None] - kpos[:, None, :]).abs().float()
        x = x - s["slopes"].view(1, hkv, 1, r, 1) * dist[:, None, :, None, :]
    p, lse = _softmax(x.masked_fill(~seen[:, None, :, None, :], -math.inf))
    out = (p.flatten(2, 3) @ v).view(n, hkv, w, r, d).permute(0, 2, 1, 3, 4).flatten(2, 3)
    lse = lse.permute(0, 2, 1, 3).flatten(2, 3)
    seq, place = pad["seq"], pad["place"]
    return out[seq, place].to(s["q"].dtype), lse[seq, place].t().contiguous()


def _plain_select(s):
    """Blocks by the bound on sum over the group's heads of q . k; 64 bits, since a choice hangs on
    the order of near values; rounded to 32 bits once, before they are compared."""
    c = s["case"]
    n, hq, d = s["q"].shape
    hkv, bs, sel = c["hkv"], c["bs"], c["select"]
    q = s["q"].double().view(n, hkv, hq // hkv, d)
    up, down = q.clamp_min(0).sum(2), q.clamp_max(0).sum(2)
    b = s["bounds"][s["table"].long()].double()  # [n, blocks, hkv, 2, d]
    x = ((b[:, :, :, 1] * up[:, None]).sum(-1) + (b[:, :, :, 0] * down[:, None]).sum(-1))
    x = x.float().permute(0, 2, 1)  # [n, hkv, blocks]
    nblk = (s["len_t"] + bs - 1) // bs
    j = torch.arange(x.shape[2], device="cuda")
    forced = (j[None, :] < 1) | (j[None, :] == nblk[:, None] - 1)
    x = x.masked_fill(forced[:, None], math.inf)
    x = x.masked_fill((j[None, :] >= nblk[:, None])[:, None], -math.inf)
    order = torch.argsort(x, dim=2, descending=True, stable=True)[:, :, :sel]
    dead = order >= nblk[:, None, None]
    big = x.shape[2]
    order = torch.where(dead, torch.full_like(order, big), order).sort(2).values
    picked = torch.where(order >= big, torch.full_like(order, -1), order).to(torch.int32)
    if picked.shape[2] < sel:
        picked = torch.nn.functional.pad(picked, (0, sel - picked.shape[2]), value=-1)
    return picked


def _plain_sparse(s):
    bs = s["case"]["bs"]
    picked = _plain_select(s)
    slot = torch.arange(bs, device="cuda")
    blk = picked.long().clamp_min(0)
    keys = (blk[..., None] * bs + slot).flatten(2)
    ids = torch.gather(s["table"].long()[:, None].expand(-1, blk.shape[1], -1), 2, blk)
    rows = (ids[..., None] * bs + slot).flatten(2)
    valid = (picked >= 0).repeat_interleave(bs, 2) & (keys < s["len_t"][:, None, None])
    p, out, lse = _plain_decode(s, rows, keys, valid)
    return picked, out, lse


def _plain_bounds(s):
    bs = s["case"]["bs"]
    nblk = (s["len_t"] + bs - 1) // bs
    first = s["first"].long() // bs if s["first"] is not None else torch.zeros_like(nblk)
    new = s["case"]["newest"]
    width = min(s["table"].shape[1], (new + bs - 2) // bs + 1) if new else s["table"].shape[1]
    j = first[:, None] + torch.arange(width, device="cuda")
    live = j < nblk[:, None]
    ids = torch.gather(s["table"].long(), 1, j.clamp_max(s["table"].shape[1] - 1))
    keys = j[:, :, None] * bs + torch.arange(bs, device="cuda")
    ids, dead = ids[live], (keys >= s["len_t"][:, None, None])[live]
    x = s["k_cache"][ids]
    lo = x.masked_fill(dead[:, :, None, None], math.inf).amin(1)
    hi = x.masked_fill(dead[:, :, None, None], -math.inf).amax(1)
    s["bounds"][ids] = torch.stack((lo, hi), 2)
    return s["bounds"]


def _plain_weights(s):
    keys = torch.arange(s["max"], device="cuda")[None, :].expand(s["case"]["n"], -1)
    p, out, lse = _plain_decode(s, s["rows"], keys, s["valid"])
    w = p.sum(2)
    if s["prev"] is not None:
        w = w + s["prev"]
    s["weights"].copy_(torch.where(s["valid"][:, None], w, s["weights"]))
    return out, lse, s["weights"]


def _plain_prompt(s):
    c, pad = s["case"], s["pad"]
    n, w, hkv = c["n"], s["max"], c["hkv"]
    r = c["hq"] // hkv
    last = min(c["last"] or w, w)
    at = torch.arange(w, device="cuda")
    # the last queries of each prompt, padded: their places in it (negative: there is none)
    place = s["len_t"][:, None] - last + torch.arange(last, device="cuda")
    live = place >= 0
    row = torch.gather(pad["row"], 1, place.clamp_min(0))
    keep = (at <= place[:, :, None]) & live[:, :, None]  # [n, last, w]
    dist = (place[:, :, None] - at).float() if s["slopes"] is not None else None
    out = s["weights"]
    for h in range(c["hq"]):  # one head at a time: all heads' scores would not fit
        q, k = s["q"][row, h].float(), s["k"][pad["row"], h // r].float()
        x = (q @ k.transpose(1, 2)) * s["scale"] - s["lse"][h][row][:, :, None]
        if dist is not None:
            x = x - s["slopes"][h] * dist
        p = torch.where(keep, torch.exp(x), torch.zeros_like(x)).sum(1)
        if h % r == 0:
            out[:, h // r] = p
        else:
            out[:, h // r] += p
    return out


def _plain_evict(s):
    c = s["case"]
    keep, recent, bs = c["keep"], c["recent"], c["bs"]
    at = torch.arange(s["max"], device="cuda")
    x = s["weights"].masked_fill((at >= s["len_t"][:, None] - recent)[:, None], math.inf)
    x = x.masked_fill(~s["valid"][:, None], -math.inf)
    order = torch.argsort(x, dim=2, descending=True, stable=True)[:, :, :keep]
    big = s["max"]
    dead = order >= s["len_t"][:, None, None]
    order = torch.where(dead, torch.full_like(order, big), order).sort(2).values
    if order.shape[2] < keep:
        order = torch.nn.functional.pad(order, (0, keep - order.shape[2]), value=big)
    dead = order >= big
    idx = order.clamp_max(big - 1)
    kept = torch.where(dead, torch.full_like(order, -1), order).to(torch.int32)
    w = torch.gather(s["weights"], 2, idx).masked_fill(dead, 0)
    s["out_weights"].copy_(w)
    t = torch.arange(keep, device="cuda")
    dst = s["out_table"].long()[:, t // bs] * bs + t % bs  # [n, keep]
    src = torch.gather(s["rows"][:, None].expand(-1, c["hkv"], -1), 2, idx)
    head = torch.arange(c["hkv"], device="cuda")[None, :, None].expand_as(src)
    dst = dst[:, None].expand_as(src)
    live = ~dead
    src, dst, head = src[live], dst[live], head[live]
    s["out_k"].flatten(0, 1)[dst, head] = s["k_cache"].flatten(0, 1)[src, head]
    s["out_v"].flatten(0, 1)[dst, head] = s["v_cache"].flatten(0, 1)[src, head]
    left = s["len_t"].clamp_max(keep)
    cu = torch.cat((torch.zeros(1, dtype=left.dtype, device="cuda"), torch.cumsum(left, 0)))
    return kept, s["out_weights"], cu.to(torch.int32), s["out_k"], s["out_v"]


PLAIN = {"tree": _plain_tree, "sparse": _plain_sparse, "bounds": _plain_bounds,
         "weights": _plain_weights, "prompt": _plain_prompt, "evict": _plain_evict}


# ------------------------------------------------------------------------------------------
# The framework's calls.
# ------------------------------------------------------------------------------------------
def _workspace(s, size):
    """A workspace of the program's, made before its first step and kept."""
    if "ws" not in s:
        s["ws"] = torch.empty(size(), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own(s):
    import memory_efficient_attention_b200 as mea

    c = s["case"]
    n, hq, hkv, d, op = c["n"], c["hq"], c["hkv"], c["d"], c["op"]
    if op == "tree":
        ws = _workspace(s, lambda: mea.decode_tree_workspace_size(hq, hkv, d))
        return mea.decode_tree_paged(
            s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu_q"], s["cu"], s["max_q"],
            s["max"], s["mask"], alibi_slopes=s["slopes"], scale=s["scale"], workspace=ws,
            out=s["out"], lse=s["lse"])
    if op == "sparse":
        ws = _workspace(s, lambda: mea.decode_selected_workspace_size(
            n, c["select"], c["bs"], hq, hkv, d))
        sel = mea.select_blocks(s["q"], s["bounds"], s["table"], s["cu"], s["max"], c["bs"],
                                c["select"], n_first=1, n_last=1, selected=s["selected"])
        out, lse = mea.decode_paged_selected(
            s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], sel,
            alibi_slopes=s["slopes"], scale=s["scale"], workspace=ws, out=s["out"], lse=s["lse"])
        return sel, out, lse
    if op == "bounds":
        return mea.block_key_bounds(s["k_cache"], s["table"], s["cu"], s["max"],
                                    first_key=s["first"], bounds=s["bounds"])
    if op == "weights":
        ws = _workspace(s, lambda: mea.decode_weights_workspace_size(n, s["total"], hq, hkv, d))
        return mea.decode_paged_weights(
            s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["max"], s["weights"],
            prev_weights=s["prev"], alibi_slopes=s["slopes"], scale=s["scale"], workspace=ws,
            total_k_bound=s["total"], out=s["out"], lse=s["lse"])
    if op == "prompt":
        return mea.attention_packed_weights(
            s["q"], s["k"], s["lse"], s["cu"], s["cu"], s["max"], s["max"], causal=True,
            alibi_slopes=s["slopes"], scale=s["scale"], last_queries=c["last"],
            weights=s["weights"])
    kept, w, cu = mea.evict_paged(
        s["k_cache"], s["v_cache"], s["table"], s["cu"], s["max"], s["weights"], c["keep"],
        c["recent"], s["out_table"], out_k_cache=s["out_k"], out_v_cache=s["out_v"],
        kept=s["kept"], out_weights=s["out_weights"], out_cu_seqlens_k=s["out_cu"])
    return kept, w, cu, s["out_k"], s["out_v"]


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------
# What one pass cannot do without.
# ------------------------------------------------------------------------------------------
def work(case):
    lens = _lens(case)
    hq, hkv, d, n, op = case["hq"], case["hkv"], case["d"], case["n"], case["op"]
    total, row = sum(lens), hkv * d * 2  # one key's (or value's) bytes over the KV heads
    if op == "tree":
        dr = _drafts(case)
        words = (max(dr) + 31) // 32
        return {"bytes": 2 * total * row + sum(dr) * (2 * hq * d * 2 + 4 * hq + 4 * words),
                "flops": 4 * d * hq * sum(x * y for x, y in zip(dr, lens))}
    if op == "sparse":
        bs = case["bs"]
        blocks = [-(-x // bs) for x in lens]
        keys = sum(min(x, case["select"] * bs) for x in lens)
        return {"bytes": 2 * row * sum(blocks) + 2 * keys * row + n * (2 * hq * d * 2 + 4 * hq) +
                4 * sum(blocks) + 4 * n * hkv * case["select"],
                "flops": 4 * d * hkv * sum(blocks) + 4 * d * hq * keys}
    if op == "bounds":
        bs, new = case["bs"], case["newest"]
        first = [max(0, x - new) // bs if new else 0 for x in lens]
        keys = sum(x - f * bs for x, f in zip(lens, first))
        blocks = sum(-(-x // bs) - f for x, f in zip(lens, first))
        return {"bytes": keys * row + blocks * (2 * row + 4), "flops": 2 * keys * hkv * d}
    if op == "weights":
        return {"bytes": 2 * total * row + 4 * total * hkv * (2 if case["prev"] else 1) +
                n * (2 * hq * d * 2 + 4 * hq), "flops": 4 * d * hq * total}
    if op == "prompt":
        last = [min(case["last"] or x, x) for x in lens]
        pairs = sum(x * y - y * (y - 1) // 2 for x, y in zip(lens, last))
        return {"bytes": total * row + sum(last) * hq * (2 * d + 4) + 4 * total * hkv,
                "flops": 2 * d * hq * pairs}
    kept = sum(min(x, case["keep"]) for x in lens)
    return {"bytes": 4 * total * hkv + kept * (4 * row + hkv * 8), "flops": total * hkv}


# ------------------------------------------------------------------------------------------
# The operators' definitions in 64 bits, one request (and head) at a time.
# ------------------------------------------------------------------------------------------
def _exact_rows(s, b):
    """Request b's keys (and values) in order, [L, hkv, d] in 64 bits."""
    bs, length = s["case"]["bs"], s["lens"][b]
    ids = s["table"][b, :-(-length // bs)].long()
    k = s["k_cache"][ids].double().flatten(0, 1)[:length]
    v = s["v_cache"][ids].double().flatten(0, 1)[:length] if "v_cache" in s else None
    return k, v


def _exact_attend(x, v):
    """Rows of scores [rows, keys] against values [keys, d]."""
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
    return p, p @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    op, hq, hkv, d = case["op"], case["hq"], case["hkv"], case["d"]
    r, sc, sl = hq // hkv, s["scale"], s["slopes"]
    f64 = dict(dtype=torch.float64, device="cuda")
    if op == "bounds":
        return None  # values of the inputs: nothing is rounded
    if op == "evict":
        return None  # copies and whole numbers
    if op == "prompt":
        out, off = torch.zeros((case["n"], hkv, s["max"]), **f64), 0
        for b, length in enumerate(s["lens"]):
            q0 = max(0, length - case["last"]) if case["last"] else 0
            i, j = torch.arange(q0, length, device="cuda"), torch.arange(length, device="cuda")
            for h in range(hq):
                k = s["k"][off:off + length, h // r].double()
                x = sc * (s["q"][off + q0:off + length, h].double() @ k.t())
                if sl is not None:
                    x -= sl[h].double() * (i[:, None] - j[None, :]).abs()
                x -= s["lse"][h, off + q0:off + length, None].double()
                x[j[None, :] > i[:, None]] = -math.inf
                out[b, h // r, :length] += x.exp_().sum(0)
            off += length
        return out
    if op == "tree":
        out, lse, off = torch.zeros(s["q"].shape, **f64), torch.zeros(s["lse"].shape, **f64), 0
        for b, length in enumerate(s["lens"]):
            k, v = _exact_rows(s, b)
            x0 = int(s["draft_t"][b])
            m = s["mask"][off:off + x0].cpu().tolist()
            tree = torch.tensor([[(row[j // 32] >> (j % 32)) & 1 for j in range(x0)] for row in m],
                                dtype=torch.bool, device="cuda")
            seen = torch.ones((x0, length), dtype=torch.bool, device="cuda")
            seen[:, length - x0:] = tree
            pos = torch.arange(length, **f64)
            pos[length - x0:] = length - x0 + tree.sum(1) - 1
            for h in range(hq):
                x = sc * (s["q"][off:off + x0, h].double() @ k[:, h // r].t())
                if sl is not None:
                    x -= sl[h].double() * (pos[length - x0:, None] - pos[None, :]).abs()
                _, o, z = _exact_attend(x.masked_fill(~seen, -math.inf), v[:, h // r])
                out[off:off + x0, h], lse[h, off:off + x0] = o, z
            off += x0
        return out, lse
    out, lse = torch.zeros(s["q"].shape, **f64), torch.zeros(s["lse"].shape, **f64)
    if op == "weights":
        w = s["weights"].double()
        for b, length in enumerate(s["lens"]):
            k, v = _exact_rows(s, b)
            back = torch.arange(length - 1, -1, -1, **f64)
            for g in range(hkv):
                x = sc * (s["q"][b, g * r:(g + 1) * r].double() @ k[:, g].t())
                if sl is not None:
                    x -= sl[g * r:(g + 1) * r, None].double() * back
                p, o, z = _exact_attend(x, v[:, g])
                out[b, g * r:(g + 1) * r], lse[g * r:(g + 1) * r, b] = o, z
                w[b, g, :length] = p.sum(0)
                if s["prev"] is not None:
                    w[b, g, :length] += s["prev"][b, g, :length]
        return out, lse, w
    bs, sel = case["bs"], case["select"]  # sparse
    for b, length in enumerate(s["lens"]):
        k, v = _exact_rows(s, b)
        nblk = -(-length // bs)
        lo, hi = s["bounds"][s["table"][b, :nblk].long()].double().unbind(2)  # [blocks, hkv, d]
        for g in range(hkv):
            q = s["q"][b, g * r:(g + 1) * r].double()
            best = torch.maximum(q[:, None] * lo[None, :, g], q[:, None] * hi[None, :, g])
            score = best.sum((0, 2)).float()
            score[0] = score[nblk - 1] = math.inf
            top = torch.sort(score, descending=True, stable=True).indices[:sel].sort().values
            keys = (top[:, None] * bs + torch.arange(bs, device="cuda")).flatten()
            keys = keys[keys < length]
            x = sc * (q @ k[keys, g].t())
            if sl is not None:
                x -= sl[g * r:(g + 1) * r, None].double() * (length - 1 - keys)
            _, o, z = _exact_attend(x, v[keys, g])
            out[b, g * r:(g + 1) * r], lse[g * r:(g + 1) * r, b] = o, z
    return None, out, lse
