"""Cases, plain forms and 64-bit values of the operators beside the packed cache.

Four operators of a serving step with head dimension 128:

  rope_pack     isoquant_decode_prep_rope: rotate keys and queries by position, compress K and V into the packed
                paged cache, isotropize the queries
  rope_dense    isoquant_dense_prep: the same step for a paged cache that keeps 16-bit keys and values
  dense_attend  isoquant_dense_attend: attention of new tokens over that cache
  prompt        isoquant_prompt_attend: attention of whole prompts, packed one after another, to themselves

`own` false: elementary torch operations.  `own` true: the library's calls.
"""
import functools
import math

import torch

own = False

D = 128
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
WORDS = {2: 8, 3: 13, 4: 16}
PER_WORD = {2: 16, 3: 10, 4: 8}


# ------------------------------------------------------------------ cases
def _pack(name, n_tok, q_heads, kv_heads, dtype="bf16", bits=3, page_size=256, rot=128, interleaved=False, skip=0):
    return {"name": name, "op": "rope_pack", "n_tok": n_tok, "q_heads": q_heads, "kv_heads": kv_heads, "dtype": dtype,
            "bits": bits, "page_size": page_size, "rot": rot, "interleaved": interleaved, "skip": skip}


def _dense(name, n_tok, q_heads, kv_heads, dtype="bf16", page_size=256, rot=128, interleaved=False, skip=0,
           k_out=False):
    return {"name": name, "op": "rope_dense", "n_tok": n_tok, "q_heads": q_heads, "kv_heads": kv_heads,
            "dtype": dtype, "page_size": page_size, "rot": rot, "interleaved": interleaved, "skip": skip,
            "k_out": k_out}


def _attend(name, lens, q_heads, kv_heads, nq=1, dtype="bf16", page_size=256, causal=False):
    return {"name": name, "op": "dense_attend", "lens": ",".join(map(str, lens)), "nq": nq, "q_heads": q_heads,
            "kv_heads": kv_heads, "dtype": dtype, "page_size": page_size, "causal": causal}


def _prompt(name, lens, q_heads, kv_heads, dtype="bf16", causal=True, tail=0):
    return {"name": name, "op": "prompt", "lens": ",".join(map(str, lens)), "q_heads": q_heads, "kv_heads": kv_heads,
            "dtype": dtype, "causal": causal, "tail": tail}


def listed():
    return [
        # one decode step of 16 sequences of a 32-query-head, 4-KV-head model: pure latency
        _pack("pack_step_b16_q32_kv4", 16, 32, 4),
        # the tokens of an 8192-token prompt entering the packed cache
        _pack("pack_prompt_8192_q32_kv8", 8192, 32, 8),
        # a padded batch (a tenth of its slots skipped), 4-bit codes, half of each head rotated in adjacent pairs
        _pack("pack_777_q4_kv1_4bit_f16", 777, 4, 1, dtype="f16", bits=4, page_size=64, rot=64, interleaved=True,
              skip=10),
        # the same decode step into 16-bit pages
        _dense("dense_step_b16_q32_kv4", 16, 32, 4),
        # a 32768-token prompt entering 16-bit pages, its rotated keys also written out for the prompt's attention
        _dense("dense_prompt_32768_q32_kv8", 32768, 32, 8, k_out=True),
        # one sequence, one head, a short context: the smallest decode call
        _attend("attend_single_head_L1024", [1024], 1, 1, dtype="f16", page_size=64),
        # a decode batch of 16 at 32768 tokens, 8 query heads per KV head
        _attend("attend_b16_q32_kv4_L32768", [32768] * 16, 32, 4),
        # four long ragged contexts of a 64-query-head model
        _attend("attend_b4_q64_kv8_ragged", [66113, 131072, 98305, 71007], 64, 8),
        # a speculative chunk of 16 tokens per sequence, each seeing its own prefix
        _attend("attend_verify_b8_nq16_L16384", [16384] * 8, 32, 8, nq=16, page_size=128, causal=True),
        # short prompts of one serving batch packed together, with padding rows behind the last
        _prompt("prompt_ragged16_q32_kv4", [1, 17, 300, 511, 64, 129, 77, 256, 33, 480, 2, 190, 401, 128, 5, 350], 32,
                4, tail=20),
        # an 8192-token prompt
        _prompt("prompt_8192_q32_kv8_f16", [8192], 32, 8, dtype="f16"),
        # a 32768-token prompt
        _prompt("prompt_32768_q32_kv8", [32768], 32, 8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope_pack", "rope_dense", "dense_attend", "prompt"])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 6, 8])
    dtype = rng.choice(["bf16", "f16"])
    page = rng.choice([32, 64, 128, 256])
    rot, inter, skip = rng.choice([32, 64, 96, 128]), rng.random() < 0.4, rng.choice([0, 0, 10, 35])
    if op == "rope_pack":
        n = _log(rng, 1, 8192)
        c = _pack("", n, kv * group, kv, rng.choice(["bf16", "f16", "f32"]), rng.choice([2, 3, 4]), page, rot, inter,
                  skip)
    elif op == "rope_dense":
        n = _log(rng, 1, min(32768, 32768 * 32 // (kv * group)))
        c = _dense("", n, kv * group, kv, dtype, page, rot, inter, skip, rng.random() < 0.5)
    elif op == "dense_attend":
        nq = rng.choice([1, 1, 1, 2, 5, 16])
        batch = _log(rng, 1, 24)
        # token x head products no more than the largest listed case's, and nq times fewer for a chunk
        top = min(131072, 2_000_000 // (kv * batch * nq))
        lens = [_log(rng, 1, top) for _ in range(batch)]
        if batch > 2 and rng.random() < 0.5:
            lens[rng.randrange(batch)] = 0
        c = _attend("", lens, kv * group, kv, nq, dtype, page, nq > 1 and rng.random() < 0.8)
    else:
        batch = _log(rng, 1, 24)
        top = max(16, int(math.sqrt(1.0e10 / (kv * group * batch))))
        lens = [_log(rng, 1, min(16384, top)) for _ in range(batch)]
        if batch > 2 and rng.random() < 0.5:
            lens[rng.randrange(batch)] = 0
        c = _prompt("", lens, kv * group, kv, dtype, rng.random() < 0.8, rng.choice([0, 0, 3, 40]))
    del c["name"]
    return c


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def work(case):
    """Bytes that have to move and operations that have to be done, each input read and each output written once."""
    op, H, Hq = case["op"], case["kv_heads"], case["q_heads"]
    if op in ("rope_pack", "rope_dense"):
        n, eb = case["n_tok"], 4 if case["dtype"] == "f32" else 2
        kept = n - n * case["skip"] // 100
        read = n * Hq * D * eb + (kept if not case.get("k_out") else n) * H * D * eb + kept * H * D * eb
        read += n * (8 + 2 * 8 + 4 * case["rot"])
        if op == "rope_pack":
            written = kept * H * 2 * (4 * WORDS[case["bits"]] + 2) + n * Hq * D * 4
            # per vector: the rotation by position, seven butterfly stages, 32 products of 4 x 4, the norm
            flops = (n * Hq + 2 * kept * H) * (7 * D + 7 * D + 2 * D) + (n * Hq + kept * H) * 3 * case["rot"]
        else:
            written = kept * H * 2 * D * 2 + n * Hq * D * 2 + (n * H * D * 2 if case["k_out"] else 0)
            flops = n * (Hq + H) * 3 * case["rot"]
        return {"bytes": read + written, "flops": flops}
    lens = _lens(case)
    if op == "dense_attend":
        nq, B = case["nq"], len(lens)
        if case["causal"]:
            pairs = sum(max(0, L - nq + i + 1) for L in lens for i in range(nq))
        else:
            pairs = nq * sum(lens)
        return {"bytes": sum(lens) * H * 2 * D * 2 + 2 * B * nq * Hq * D * 2, "flops": 4 * D * Hq * pairs}
    pairs = sum(L * (L + 1) // 2 if case["causal"] else L * L for L in lens)
    return {"bytes": sum(lens) * D * 2 * (2 * Hq + 2 * H), "flops": 4 * D * Hq * pairs}


# ----------------------------------------------------------------- inputs
@functools.lru_cache(maxsize=None)
def _codebook(bits):
    """Lloyd-Max levels of N(0,1) rounded to fp16 and the midpoints between them (64-bit)."""
    n = 1 << bits
    pdf = lambda z: math.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)  # noqa: E731
    cdf = lambda z: 0.5 * math.erfc(-z / math.sqrt(2))  # noqa: E731
    lv = [3.0 * (2 * i + 1 - n) / n for i in range(n)]
    for _ in range(20000):
        th = [-math.inf] + [(a + b) / 2 for a, b in zip(lv, lv[1:])] + [math.inf]
        new = [((pdf(a) if a > -math.inf else 0.0) - (pdf(b) if b < math.inf else 0.0)) / (cdf(b) - cdf(a))
               for a, b in zip(th, th[1:])]
        moved = max(abs(a - b) for a, b in zip(new, lv))
        lv = new
        if moved < 1e-13:
            break
    lv = torch.tensor(lv, dtype=torch.float64).to(torch.float16).to(torch.float64)
    return lv, (lv[1:] + lv[:-1]) / 2


def _rotation_matrices(signs, quats):
    """R = B Hn D of every head, 64-bit [H][128][128]: signs, Sylvester matrix / sqrt(128), 32 blocks
    v -> qL v conj(qR) written as 4 x 4 matrices."""
    H = signs.shape[0]
    had = torch.ones((1, 1), dtype=torch.float64)
    for _ in range(7):
        had = torch.cat([torch.cat([had, had], 1), torch.cat([had, -had], 1)], 0)
    had = had / math.sqrt(D)
    q = quats.double()
    q = q / q.norm(dim=-1, keepdim=True)
    a, b, c, d = q[:, :, 0].unbind(-1)
    left = torch.stack([a, -b, -c, -d, b, a, -d, c, c, d, a, -b, d, -c, b, a], -1).view(H, 32, 4, 4)
    a, b, c, d = (q[:, :, 1] * torch.tensor([1.0, -1, -1, -1], dtype=torch.float64)).unbind(-1)
    right = torch.stack([a, -b, -c, -d, b, a, d, -c, c, -d, a, b, d, c, -b, a], -1).view(H, 32, 4, 4)
    blocks = torch.zeros((H, D, D), dtype=torch.float64)
    at = torch.arange(32)
    m = left @ right
    for i in range(4):
        for j in range(4):
            blocks[:, 4 * at + i, 4 * at + j] = m[:, :, i, j]
    return blocks @ (had[None] * signs.double()[:, None, :])


def _rope_table(n, rot):
    """[n][rot]: the cosines of position x base^(-2i/rot), i < rot/2, then the sines; angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    ang = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * inv[None]
    return torch.cat([torch.cos(ang), torch.sin(ang)], 1).to(torch.float32)


def _scales(g, heads):
    """Channel scales of keys and values, log-uniform in [0.4, 2.5]."""
    return torch.exp((torch.rand((heads, D), generator=g, device="cuda") - 0.5) * (2 * math.log(2.5)))


def _normal(g, shape, dtype, scale=None):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return (x if scale is None else x.mul_(scale)).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 13)
    hg = torch.Generator()
    hg.manual_seed(seed * 104729 + 7)
    dt, H, Hq, op = DTYPES[case["dtype"]], case["kv_heads"], case["q_heads"], case["op"]
    s = {"case": case}
    signs = (torch.randint(0, 2, (H, D), generator=hg) * 2 - 1).to(torch.int8)
    quats = torch.randn((H, 32, 2, 4), generator=hg)
    if own:
        import compressed_space_decode_b200 as csd
        s["lib"] = csd
        s["ctx"] = csd.isoquant_init(signs, quats, bits=case.get("bits", 3))
    if op in ("rope_pack", "rope_dense"):
        n, ps = case["n_tok"], case["page_size"]
        far = 40000
        s["table"] = _rope_table(far + n, case["rot"])
        s["k"] = _normal(g, (n, H, D), dt, _scales(g, H))
        s["v"] = _normal(g, (n, H, D), dt, _scales(g, H))
        s["q"] = _normal(g, (n, Hq, D), dt)
        if n <= 64:  # a decode step: sequences at positions of their own
            s["pos"] = torch.randint(1000, far, (n,), generator=g, device="cuda")
        else:  # consecutive tokens of a prompt
            first = int(torch.randint(0, far, (1,), generator=hg))
            s["pos"] = torch.arange(first, first + n, device="cuda")
        pages = max(4, -(-n // ps)) if n > 64 else max(4, n)
        order = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(n, device="cuda")
        if n > 64:
            slots = order[t // ps] * ps + t % ps
        else:  # each token in its own page
            slots = order[t] * ps + torch.randint(0, ps, (n,), generator=g, device="cuda")
        drop = n * case["skip"] // 100
        slots[torch.randperm(n, generator=g, device="cuda")[:drop]] = -1
        s["slots"] = slots
        if op == "rope_pack":
            bits = case["bits"]
            s["codes"] = torch.randint(-2**31, 2**31 - 1, (pages, 2, H, WORDS[bits], ps), generator=g, device="cuda",
                                       dtype=torch.int32)
            s["norms"] = _normal(g, (pages, 2, H, ps), torch.float16)
            s["signs"], s["quats"] = signs, quats
            s["R"] = _rotation_matrices(signs, quats).cuda()
            s["thresholds"] = _codebook(bits)[1].cuda()
            s["q_rot"] = torch.empty((n, Hq, D), dtype=torch.float32, device="cuda")
            if own:
                s["cache"] = csd.PagedCache(s["codes"], s["norms"], ps)
        else:
            s["data"] = _normal(g, (pages, 2, H, ps, D), dt)
            s["q_out"] = torch.empty((n, Hq, D), dtype=dt, device="cuda")
            s["k_out"] = torch.empty((n, H, D), dtype=dt, device="cuda") if case["k_out"] else None
            if own:
                s["cache"] = csd.DenseCache(s["data"], ps)
        if own:
            s["rope"] = csd.Rope(s["table"], case["rot"], case["interleaved"])
        return s
    lens = _lens(case)
    B = len(lens)
    s["lens"] = lens
    if op == "dense_attend":
        ps, nq = case["page_size"], case["nq"]
        per = [max(1, -(-L // ps)) for L in lens]
        order = torch.randperm(sum(per), generator=hg).to(torch.int32)
        table = torch.zeros((B, max(per)), dtype=torch.int32)
        at = 0
        for b, m in enumerate(per):
            table[b, :m] = order[at:at + m]
            at += m
        s["page_table"] = table.cuda()
        data = torch.empty((sum(per), 2, H, ps, D), dtype=dt, device="cuda")
        data.normal_(generator=g)
        data[:, 0] *= _scales(g, H)[:, None].to(dt)
        data[:, 1] *= _scales(g, H)[:, None].to(dt)
        s["data"] = data
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = _normal(g, (B, nq, Hq, D), dt)
        s["out"] = torch.empty((B, nq, Hq, D), dtype=dt, device="cuda")
        if own:
            s["cache"] = csd.DenseCache(data, ps)
            s["ws"] = csd.alloc_dense_workspace(s["ctx"], B, nq, Hq)
        return s
    T = sum(lens) + case["tail"]
    s["q"] = _normal(g, (T, Hq, D), dt)
    s["k"] = _normal(g, (T, H, D), dt, _scales(g, H))
    s["v"] = _normal(g, (T, H, D), dt, _scales(g, H))
    cu = [0]
    for L in lens:
        cu.append(cu[-1] + L)
    s["cu"] = cu
    s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["out"] = _normal(g, (T, Hq, D), dt)  # the rows behind the last sequence stay as they are
    return s


# ------------------------------------------------------------ plain forms
def _rotate(x, cos, sin, rot, interleaved):
    """The position rotation of x [n][heads][128]; cos, sin [n][rot / 2]; in x's type."""
    c, sn = cos[:, None], sin[:, None]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * c - b * sn
        y[..., 1:rot:2] = b * c + a * sn
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * c - b * sn
        y[..., rot // 2:rot] = b * c + a * sn
    return y


def _plain_pack(s):
    c = s["case"]
    rot, inter, bits, ps = c["rot"], c["interleaved"], c["bits"], c["page_size"]
    at = s["table"][s["pos"]]
    cos, sin = at[:, :rot // 2], at[:, rot // 2:]
    G = c["q_heads"] // c["kv_heads"]
    q = _rotate(s["q"].float(), cos, sin, rot, inter)
    R32 = s["R"].float().repeat_interleave(G, 0)
    s["q_rot"].copy_(torch.einsum("hij,nhj->nhi", R32, q))
    # codes in 64 bits: a coordinate next to a threshold decides a whole step
    keep = s["slots"] >= 0
    slots = s["slots"][keep]
    k = _rotate(s["k"].double(), cos.double(), sin.double(), rot, inter)
    kv = torch.stack([k, s["v"].double()], 1)[keep]  # [n][2][H][128]
    norm = (kv * kv).sum(-1).sqrt()
    z = torch.einsum("hij,nkhj->nkhi", s["R"], kv) * math.sqrt(D)
    z = torch.where(norm[..., None] > 0, z / norm[..., None], torch.zeros_like(z))
    code = (z[..., None] > s["thresholds"]).sum(-1)
    W, per = WORDS[bits], PER_WORD[bits]
    code = torch.cat([code, code.new_zeros(code.shape[:-1] + (W * per - D,))], -1).view(code.shape[:-1] + (W, per))
    words = (code << (bits * torch.arange(per, device="cuda"))).sum(-1)
    words = torch.where(words >= 2**31, words - 2**32, words).to(torch.int32)
    page, off = slots // ps, slots % ps
    s["codes"].permute(0, 4, 1, 2, 3)[page, off] = words
    s["norms"].permute(0, 3, 1, 2)[page, off] = norm.clamp(max=65504.0).to(torch.float16)
    return {"codes": s["codes"], "norms": s["norms"], "q_rot": s["q_rot"]}


def _plain_dense(s):
    c = s["case"]
    rot, inter, ps = c["rot"], c["interleaved"], c["page_size"]
    at = s["table"][s["pos"]]
    cos, sin = at[:, :rot // 2], at[:, rot // 2:]
    s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, rot, inter))
    k = _rotate(s["k"].float(), cos, sin, rot, inter).to(s["data"].dtype)
    if s["k_out"] is not None:
        s["k_out"].copy_(k)
    keep = s["slots"] >= 0
    slots = s["slots"][keep]
    s["data"].permute(0, 3, 1, 2, 4)[slots // ps, slots % ps] = torch.stack([k, s["v"]], 1)[keep]
    out = {"data": s["data"], "q_out": s["q_out"]}
    if s["k_out"] is not None:
        out["k_out"] = s["k_out"]
    return out


def _softmax_rows(scores, seen, v):
    """softmax(scores where seen) v, zeros for a row that sees nothing; 32 bits."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total > 0, total, torch.ones_like(total))


def _plain_attend(s):
    c = s["case"]
    H, Hq, nq, ps = c["kv_heads"], c["q_heads"], c["nq"], c["page_size"]
    G, B = Hq // H, s["q"].shape[0]
    held = s["data"][s["page_table"].long()]  # [B][pages][2][H][ps][128]
    T = held.shape[1] * ps
    lens = s["seq_lens"].long()
    t = torch.arange(T, device="cuda")
    k = held[:, :, 0].permute(0, 2, 1, 3, 4).reshape(B, H, T, D).float()
    v = held[:, :, 1].permute(0, 2, 1, 3, 4).reshape(B, H, T, D).float()
    v = v.masked_fill(~(t < lens[:, None])[:, None, :, None], 0.0)
    q = s["q"].float().view(B, nq, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, nq * G, D)
    limit = lens[:, None].expand(B, nq)
    if c["causal"]:
        limit = lens[:, None] - nq + torch.arange(nq, device="cuda") + 1
    seen = (t < limit[..., None])[:, None, :, None].expand(B, 1, nq, G, T).reshape(B, 1, nq * G, T)
    o = _softmax_rows((q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(D)), seen, v)
    s["out"].copy_(o.view(B, H, nq, G, D).permute(0, 2, 1, 3, 4).reshape(B, nq, Hq, D))
    return s["out"]


def _plain_prompt(s):
    c = s["case"]
    H, Hq, causal = c["kv_heads"], c["q_heads"], c["causal"]
    G = Hq // H
    for a, b in zip(s["cu"], s["cu"][1:]):
        k = s["k"][a:b].float().permute(1, 2, 0)
        v = s["v"][a:b].float().transpose(0, 1)
        step = max(1, min(1024, 2**28 // max(1, (b - a) * Hq)))  # the scores of a whole prompt do not fit
        for i in range(a, b, step):
            j = min(i + step, b)
            end = j - a if causal else b - a
            q = s["q"][i:j].float().view(j - i, H, G, D).permute(1, 2, 0, 3).reshape(H, G * (j - i), D)
            seen = torch.ones((j - i, end), dtype=torch.bool, device="cuda")
            if causal:
                seen = seen.tril(i - a)
            o = _softmax_rows((q @ k[:, :, :end]) * (1.0 / math.sqrt(D)), seen.repeat(G, 1), v[:, :end])
            s["out"][i:j] = o.view(H, G, j - i, D).permute(2, 0, 1, 3).reshape(j - i, Hq, D).to(s["out"].dtype)
    return s["out"]


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"rope_pack": _plain_pack, "rope_dense": _plain_dense, "dense_attend": _plain_attend,
                "prompt": _plain_prompt}[op](s)
    lib = s["lib"]
    if op == "rope_pack":
        lib.isoquant_decode_prep_rope(s["ctx"], s["cache"], s["k"], s["v"], s["slots"], s["pos"], s["q"], s["pos"],
                                      s["rope"], s["q_rot"])
        return {"codes": s["codes"], "norms": s["norms"], "q_rot": s["q_rot"]}
    if op == "rope_dense":
        lib.isoquant_dense_prep(s["ctx"], s["cache"], s["k"], s["v"], s["slots"], s["pos"], s["q"], s["pos"],
                                s["rope"], s["q_out"], k_out=s["k_out"])
        out = {"data": s["data"], "q_out": s["q_out"]}
        if s["k_out"] is not None:
            out["k_out"] = s["k_out"]
        return out
    if op == "dense_attend":
        lib.isoquant_dense_attend(s["ctx"], s["cache"], s["q"], s["page_table"], s["seq_lens"], s["ws"], s["out"],
                                  causal=c["causal"])
        return s["out"]
    lib.isoquant_prompt_attend(s["ctx"], s["q"], s["k"], s["v"], s["cu_seqlens"], s["out"], causal=c["causal"])
    return s["out"]


# ---------------------------------------------------------- 64-bit values
def _exact_rope(x, pos, table, rot, interleaved):
    """Each pair as a complex number times cos + i sin of its position, in 64 bits."""
    w = torch.complex(table[pos, :rot // 2].double(), table[pos, rot // 2:].double())[:, None]
    x = x.double()
    if interleaved:
        y = torch.view_as_complex(x[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * w
        y = torch.view_as_real(y).flatten(-2)
    else:
        y = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * w
        y = torch.cat([y.real, y.imag], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _exact_isotropize(x, signs, quats):
    """B Hn D x of x [n][H][128], by butterflies and quaternion products."""
    y = x * signs.to(x.device).double()
    n, H = y.shape[:2]
    for i in range(7):
        y = y.reshape(n, H, D >> (i + 1), 2, 1 << i)
        y = torch.stack([y[:, :, :, 0] + y[:, :, :, 1], y[:, :, :, 0] - y[:, :, :, 1]], 3)
    y = y.reshape(n, H, 32, 4) / math.sqrt(D)

    def times(a, b):
        aw, ax, ay, az = a.unbind(-1)
        bw, bx, by, bz = b.unbind(-1)
        return torch.stack([aw * bw - ax * bx - ay * by - az * bz, aw * bx + ax * bw + ay * bz - az * by,
                            aw * by - ax * bz + ay * bw + az * bx, aw * bz + ax * by - ay * bx + az * bw], -1)

    u = quats.to(x.device).double()
    u = u / u.norm(dim=-1, keepdim=True)
    conj = u[:, :, 1] * torch.tensor([1.0, -1, -1, -1], dtype=torch.float64, device=x.device)
    return times(times(u[:, :, 0].expand(n, H, 32, 4), y), conj.expand(n, H, 32, 4)).reshape(n, H, D)


def _exact_rows(q, k, v, limits):
    """softmax(q k / sqrt(128)) v over the first limits[r] tokens of each row; q [H][R][128], k, v [H][T][128]."""
    sc = torch.matmul(q, k.transpose(1, 2)) / math.sqrt(D)
    hide = torch.arange(k.shape[1], device="cuda")[None] >= limits[:, None]
    p = torch.softmax(sc.masked_fill_(hide[None], -math.inf), -1)
    return torch.matmul(p.nan_to_num_(0.0), v)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, H, Hq = case["op"], case["kv_heads"], case["q_heads"]
    G = Hq // H
    if op in ("rope_pack", "rope_dense"):
        rot, inter, ps = case["rot"], case["interleaved"], case["page_size"]
        k = _exact_rope(s["k"], s["pos"], s["table"], rot, inter)
        q = _exact_rope(s["q"], s["pos"], s["table"], rot, inter)
        page, off = s["slots"].div(ps, rounding_mode="floor"), s["slots"] % ps
        live = (s["slots"] >= 0).nonzero()[:, 0]
        page, off = page[live], off[live]
        if op == "rope_pack":
            norms = s["norms"].double()
            for side, x in ((0, k), (1, s["v"].double())):
                norms[page, side, :, off] = torch.linalg.vector_norm(x[live], dim=-1)
            n = q.shape[0]
            grouped = q.view(n, H, G, D).transpose(1, 2).reshape(n * G, H, D)
            q_rot = _exact_isotropize(grouped, s["signs"], s["quats"]).view(n, G, H, D).transpose(1, 2)
            return {"codes": None, "norms": norms, "q_rot": q_rot.reshape(n, Hq, D)}
        data = s["data"].double()
        data[page, 0, :, off] = k[live]
        data[page, 1, :, off] = s["v"].double()[live]
        out = {"data": data, "q_out": q}
        if case["k_out"]:
            out["k_out"] = k
        return out
    if op == "dense_attend":
        ps, nq = case["page_size"], case["nq"]
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for b, L in enumerate(s["lens"]):
            if L == 0:
                continue
            held = s["data"][s["page_table"][b, :-(-L // ps)].long()].transpose(0, 2)  # [H][2][pages][ps][128]
            kv = held.reshape(H, 2, -1, D)[:, :, :L]
            at = torch.arange(nq, device="cuda").repeat_interleave(G)
            limits = (L - nq + 1 + at) if case["causal"] else torch.full_like(at, L)
            rows = s["q"][b].double().view(nq, H, G, D).transpose(0, 1).reshape(H, nq * G, D)
            for h in range(H):
                o = _exact_rows(rows[h:h + 1], kv[h:h + 1, 0].double(), kv[h:h + 1, 1].double(), limits)
                out[b, :, h * G:(h + 1) * G] = o.view(nq, G, D)
        return out
    out = s["out"].double()
    for b, L in enumerate(s["lens"]):
        a = s["cu"][b]
        for h in range(H):
            k, v = s["k"][a:a + L, h].double()[None], s["v"][a:a + L, h].double()[None]
            for i in range(0, L, 4096):
                j = min(L, i + 4096)
                end = j if case["causal"] else L
                rows = s["q"][a + i:a + j, h * G:(h + 1) * G].double().transpose(0, 1)  # [G][n][128]
                limits = torch.arange(i + 1, j + 1, device="cuda") if case["causal"] else \
                    torch.full((j - i,), L, device="cuda")
                o = _exact_rows(rows, k[:, :end], v[:, :end], limits)
                out[a + i:a + j, h * G:(h + 1) * G] = o.transpose(0, 1)
    return out
