"""Measured cases of the standalone training operators: attention with a learned relative position
bias (forward, and the backward that recomputes the probabilities and yields the bias table's
gradient) and the global gradient norm with clipping.

Attention, per sequence b and head h, with scale c = 1/sqrt(d):
  S_ij = c q_i . k_j + T[bucket(j - i), h] + mask_bj       (a mask value <= -1e30 removes the key)
  P = softmax_j(S),  O = P V,  lse_i = log sum_j exp(S_ij)  (no key left: O = 0, lse = +inf)
and, from dO and the stored O and lse,
  P_ij = exp(S_ij - lse_i),  D_i = dO_i . O_i,  dS_ij = P_ij (dO_i . v_j - D_i),
  dQ = c dS K,  dK = c dS^T Q,  dV = P^T dO,  dT[u, h] = sum of dS_ij over b and bucket(j - i) = u.
bucket() is the two-sided logarithmic one: half of the buckets for keys behind the query, half for
keys ahead; in each half the first half are exact distances, the rest grow geometrically up to
max_distance, beyond which every distance shares the last.

Clipping: norm = sqrt(sum over all tensors of g^2); out = g * min(1, max_norm / (norm + 1e-6)).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
MASKED = -1e30


# ------------------------------------------------------------------ cases
def _attn(name, op, dtype, batch, seq, heads, dim, lo=0, buckets=32, distance=128, empty=False):
    """lo: shortest valid length of a padded batch (0: no mask); empty: the first sequence has no valid key."""
    return {"name": name, "op": op, "dtype": dtype, "batch": batch, "seq": seq, "heads": heads, "dim": dim, "lo": lo,
            "buckets": buckets, "distance": distance, "empty": empty}


def listed():
    return [
        # the smallest layer the framework is tested with: latency of one call
        _attn("fwd-tiny-f32", "fwd", "f32", 2, 16, 4, 16),
        # BERT-base batch with padding
        _attn("fwd-base-bf16", "fwd", "bf16", 8, 128, 12, 64, lo=64),
        # the headline layer: B64 S128, 16 heads
        _attn("fwd-large-f16", "fwd", "f16", 64, 128, 16, 64),
        # long sequences, padded
        _attn("fwd-long-bf16", "fwd", "bf16", 4, 2048, 16, 64, lo=1024),
        # odd length and head dim, a sequence without any valid key, many far buckets
        _attn("fwd-odd-bf16", "fwd", "bf16", 3, 777, 5, 80, lo=100, buckets=64, distance=300, empty=True),
        # training: the headline layer, the stack's S512 micro-batch, the long layer, an odd one with wide heads
        _attn("bwd-large-f16", "bwd", "f16", 64, 128, 16, 64),
        _attn("bwd-stack-f16", "bwd", "f16", 16, 512, 16, 64, lo=256),
        _attn("bwd-long-bf16", "bwd", "bf16", 4, 2048, 16, 64, lo=1024),
        _attn("bwd-odd-f16", "bwd", "f16", 2, 1001, 6, 128, lo=333, buckets=48, distance=200),
        # one small layer's twelve gradients: latency
        {"name": "clip-layer-f32", "op": "clip", "dtype": "f32", "hidden": 256, "ffn": 1024, "layers": 1, "limit": 1.0},
        # every gradient of the 24-layer BERT-Large stack (288 tensors, 302 M values)
        {"name": "clip-stack-f32", "op": "clip", "dtype": "f32", "hidden": 1024, "ffn": 4096, "layers": 24, "limit": 1.0},
        # 16-bit gradients of odd sizes (a rank's ragged shards), norm below the limit: nothing is scaled
        {"name": "clip-odd-bf16", "op": "clip", "dtype": "bf16", "hidden": 497, "ffn": 1731, "layers": 9, "limit": 1e9},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "clip"])
    if op == "clip":
        layers = _log_int(rng, 1, 24)
        hidden = _log_int(rng, 16, 1024)
        ffn = min(4096, _log_int(rng, hidden, 4 * hidden))
        return {"op": op, "dtype": rng.choice(["f32", "f32", "f16", "bf16"]), "hidden": hidden, "ffn": ffn,
                "layers": layers, "limit": rng.choice([1.0, 1.0, 0.1, 1e9])}
    dtype = rng.choice(["f16", "bf16", "f16", "bf16", "f32"])
    most = 4 * 16 * 2048 * 2048 * 64
    if dtype == "f32":
        most //= 64
        dim = rng.choice([16, 32, 64, 128])
        seq = _log_int(rng, 1, 1024)
    else:
        dim = rng.choice([16, 32, 64, 64, 64, 80, 96, 128])
        seq = _log_int(rng, 1, 4096)
    heads = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    pairs = seq * seq * max(dim, 64)
    batch = max(1, min(_log_int(rng, 1, 64), most // (heads * pairs)))
    heads = max(1, min(heads, most // (batch * pairs)))
    buckets = rng.choice([8, 16, 32, 32, 64, 128])
    c = _attn("", op, dtype, batch, seq, heads, dim, lo=rng.choice([0, max(1, seq // 2), 1]), buckets=buckets,
              distance=rng.choice([64, 128, 128, 300, 1024]), empty=batch > 1 and rng.random() < 0.2)
    if c["distance"] <= buckets // 4:
        c["distance"] = 128
    if c["empty"] and not c["lo"]:
        c["lo"] = 1
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _grad_sizes(case):
    h, f = case["hidden"], case["ffn"]
    return [(3 * h, h), (3 * h,), (h, h), (h,), (h,), (h,), (f, h), (f,), (h, f), (h,), (h,), (h,)] * case["layers"]


def _views(flat, sizes):
    return [t.view(s) for t, s in zip(flat.split([math.prod(s) for s in sizes]), sizes)]


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    if case["op"] == "clip":
        # flat buffers with one view per tensor, as the data-parallel exchange keeps them
        sizes = _grad_sizes(case)
        flat = torch.empty(sum(math.prod(s) for s in sizes), dtype=dt, device="cuda").normal_(0.0, 0.02, generator=g)
        out = torch.empty_like(flat)
        return {"case": case, "flat": flat, "grads": _views(flat, sizes), "out": out, "outs": _views(out, sizes)}
    b, s, n, d = case["batch"], case["seq"], case["heads"], case["dim"]
    # Q, K and V as the packed projection leaves them: one (B, S, 3, heads, d) buffer
    qkv = torch.empty(b, s, 3, n, d, dtype=dt, device="cuda").normal_(generator=g)
    table = torch.empty(case["buckets"], n, dtype=dt, device="cuda").normal_(generator=g)
    mask = None
    if case["lo"]:
        lens = torch.randint(case["lo"], s + 1, (b,), generator=g, device="cuda")
        if case["empty"]:
            lens[0] = 0
        mask = torch.where(torch.arange(s, device="cuda")[None] < lens[:, None], 0.0, -math.inf)
    st = {"case": case, "qkv": qkv, "table": table, "mask": mask}
    if case["op"] == "bwd":
        # the forward's saved output and row statistics, and the gradient that comes back
        st["o"], st["lse"] = _forward(st)
        st["do"] = torch.empty(b, s, n, d, dtype=dt, device="cuda").normal_(generator=g)
        st["dqkv"] = torch.empty_like(qkv)
    return st


# ------------------------------------------------------------------ plain forms
def _buckets(s, buckets, distance):
    """bucket(x - (s - 1)) for x = 0 .. 2 s - 2 (key minus query position)."""
    rel = torch.arange(-(s - 1), s, device="cuda", dtype=torch.float64)
    half = buckets // 2
    exact_ = half // 2
    n = rel.abs()
    far = exact_ + torch.floor(torch.log(n.clamp(min=1) / exact_) / math.log(distance / exact_) * (half - exact_) + 1e-9)
    return (torch.where(n < exact_, n, far.clamp(max=half - 1)) + half * (rel > 0)).long()


def _scores(st):
    c, qkv = st["case"], st["qkv"].float()
    s = c["seq"]
    q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    x = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(c["dim"]))
    pos = torch.arange(s, device="cuda")
    diag = st["table"].float()[_buckets(s, c["buckets"], c["distance"])]      # (2 s - 1, heads)
    x = x + diag[pos[None, :] - pos[:, None] + s - 1].permute(2, 0, 1)
    if st["mask"] is not None:
        x = torch.where(st["mask"] <= MASKED, -math.inf, st["mask"])[:, None, None] + x
    return x, q, k, v


def _forward(st):
    x, q, k, v = _scores(st)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = torch.where(total > 0, m + torch.log(total), math.inf)
    return o.transpose(1, 2).to(st["qkv"].dtype), lse[..., 0]


def _backward(st):
    c, dt = st["case"], st["qkv"].dtype
    s, scale = c["seq"], 1.0 / math.sqrt(c["dim"])
    x, q, k, v = _scores(st)
    o, do = st["o"].float().transpose(1, 2), st["do"].float().transpose(1, 2)
    p = torch.exp(x - st["lse"][..., None])
    ds = p * (torch.matmul(do, v.transpose(2, 3)) - (do * o).sum(-1, keepdim=True))
    dv = torch.matmul(p.transpose(2, 3), do)
    dq = torch.matmul(ds, k) * scale
    dk = torch.matmul(ds.transpose(2, 3), q) * scale
    # diagonal sums: rows padded to 2 s and re-read 2 s - 1 wide put each diagonal into a column
    z = ds.double().sum(0)
    z = torch.nn.functional.pad(z.flip(1), (0, s)).reshape(c["heads"], -1)[:, :s * (2 * s - 1)].reshape(c["heads"], s, 2 * s - 1)
    z = z.sum(1)                                                             # (heads, 2 s - 1), key minus query ascending
    hot = (_buckets(s, c["buckets"], c["distance"])[:, None] == torch.arange(c["buckets"], device="cuda")).double()
    dtable = torch.matmul(z, hot).t().float().contiguous()
    return {"dq": dq.transpose(1, 2).to(dt), "dk": dk.transpose(1, 2).to(dt), "dv": dv.transpose(1, 2).to(dt), "dtable": dtable}


def _clip(st):
    grads = st["grads"]
    total = torch.stack([t.double().square().sum() for t in grads]).sum()
    norm = total.sqrt()
    coef = torch.clamp(st["case"]["limit"] / (norm + 1e-6), max=1.0).float()
    return {"norm": norm.float().reshape(1), "out": torch.cat([(t.float() * coef).to(t.dtype).reshape(-1) for t in grads])}


def _own(st):
    import transformer_layer_pre_b200 as tlp
    c = st["case"]
    if c["op"] == "clip":
        norm = tlp.clip_grad_norm(st["grads"], c["limit"], out=st["outs"])
        return {"norm": norm, "out": st["out"]}
    q, k, v = st["qkv"].unbind(2)
    if c["op"] == "fwd":
        o, lse = tlp.attention_forward(q, k, v, mask=st["mask"], bias_table=st["table"], max_distance=c["distance"])
        return {"o": o, "lse": lse}
    dq, dk, dv = st["dqkv"].unbind(2)
    dtable = tlp.attention_backward(q, k, v, st["o"], st["lse"], st["do"], mask=st["mask"], bias_table=st["table"],
                                    max_distance=c["distance"], dq=dq, dk=dk, dv=dv)[3]
    return {"dq": dq, "dk": dk, "dv": dv, "dtable": dtable}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "clip":
        return _clip(state)
    if op == "fwd":
        o, lse = _forward(state)
        return {"o": o, "lse": lse}
    return _backward(state)


# ------------------------------------------------------------------ accounting
def work(case):
    size = torch.finfo(DTYPES[case["dtype"]]).bits // 8
    if case["op"] == "clip":
        n = sum(math.prod(s) for s in _grad_sizes(case))
        return {"bytes": 2 * n * size + 4, "flops": 3 * n}
    b, s, n, d = case["batch"], case["seq"], case["heads"], case["dim"]
    act, rows = b * s * n * d * size, b * s * n * 4
    small = case["buckets"] * n * size + (b * s * 4 if case["lo"] else 0)
    valid = s * ((s + case["lo"]) / 2 if case["lo"] else s)      # query-key pairs of a sequence, on average
    if case["op"] == "fwd":
        return {"bytes": 4 * act + rows + small, "flops": 4 * b * n * valid * d}
    return {"bytes": 8 * act + rows + small + case["buckets"] * n * 4, "flops": 10 * b * n * valid * d}


# ------------------------------------------------------------------ 64 bits
def _exact_bucket(rel, buckets, distance):
    side, n = (buckets // 2 if rel > 0 else 0), abs(rel)
    half, first = buckets // 2, buckets // 4
    if n < first:
        return side + n
    # the last step k whose border first * (distance / first)^(k / steps) is not beyond n, in whole numbers
    steps = half - first
    k = 0
    while k + 1 < steps and n ** steps >= first ** (steps - k - 1) * distance ** (k + 1):
        k += 1
    return side + first + k


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "clip":
        total = math.fsum(float(torch.linalg.vector_norm(t.double())) ** 2 for t in st["grads"])
        norm = math.sqrt(total)
        coef = min(1.0, case["limit"] / (norm + 1e-6))
        return {"norm": torch.tensor([norm], dtype=torch.float64), "out": st["flat"].double() * coef}
    b, s, n, d = case["batch"], case["seq"], case["heads"], case["dim"]
    scale = d ** -0.5
    ids = torch.tensor([_exact_bucket(r, case["buckets"], case["distance"]) for r in range(-(s - 1), s)], device="cuda")
    at = (torch.arange(s, device="cuda")[None, :] - torch.arange(s, device="cuda")[:, None]) + (s - 1)
    ids = ids[at]                                                            # (s, s)
    tab = st["table"].double()
    out = {k: [] for k in (("o", "lse") if case["op"] == "fwd" else ("dq", "dk", "dv"))}
    dtab = torch.zeros(case["buckets"], n, dtype=torch.float64, device="cuda")
    for i in range(b):
        q, k, v = (st["qkv"][i, :, j].double().permute(1, 0, 2) for j in range(3))
        x = torch.einsum("hid,hjd->hij", q, k) * scale + tab.t()[:, ids]
        if st["mask"] is not None:
            m = st["mask"][i].double()
            x = (x + m).masked_fill(m <= MASKED, -math.inf)
        if case["op"] == "fwd":
            lse = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None])
            out["o"].append(torch.einsum("hij,hjd->ihd", p, v))
            out["lse"].append(torch.where(lse == -math.inf, math.inf, lse))
            continue
        o, do = st["o"][i].double(), st["do"][i].double()
        p = torch.exp(x - st["lse"][i].double()[..., None])
        delta = torch.einsum("ihd,ihd->hi", o, do)
        ds = p * (torch.einsum("ihd,hjd->hij", do, v) - delta[..., None])
        out["dq"].append(torch.einsum("hij,hjd->ihd", ds, k) * scale)
        out["dk"].append(torch.einsum("hij,hid->jhd", ds, q) * scale)
        out["dv"].append(torch.einsum("hij,ihd->jhd", p, do))
        for r in range(case["buckets"]):
            dtab[r] += torch.where(ids == r, ds, 0.0).sum((1, 2))
    res = {k: torch.stack(v) for k, v in out.items()}
    if case["op"] == "bwd":
        res["dtable"] = dtab
    return res

