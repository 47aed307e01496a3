"""Cases of the operators of an owner that holds a vocabulary table: the log
probabilities its output head gives, their gradient, and the AdamW step with
moments in 8 bits.

Operators (field "op" of a case):

  logp     per row of x the log probability of a given token under
           softmax(scale * x table^T), the distribution's entropy and its k
           likeliest tokens; "shards" cuts the table into that many tensors;
  grad     from the gradients of log probability and entropy those of x and of
           the table;
  step8    the AdamW step with a factor on the gradients, moments in 8 bits;
  moments  moments in 32 bits into the 8-bit state and back out of it.

``run`` computes a case in plain torch operations, or through the package
where ``own`` is true.  ``exact`` computes it in 64 bits from the definition.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "i32": torch.int32, "i64": torch.int64}
ADAM = dict(lr=1e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
GROUP = 128  # elements that share a scale
ALIGN = 256


def listed():
    return [
        # one token of one sequence of GPT-2-small, its 5 likeliest successors: latency
        dict(name="logp-one", op="logp", rows=50257, cols=768, n=1, table="bf16", x="bf16", ids="i64", scale=1.0,
             top=5, shards=1, pad=0.0),
        # one decoding step of 32 sequences over the Llama-3-8B head, at a temperature
        dict(name="logp-decode", op="logp", rows=128256, cols=4096, n=32, table="bf16", x="bf16", ids="i64",
             scale=1.25, top=8, shards=1, pad=0.0),
        # a small fp32 vocabulary of odd sizes, cut into two owners' tensors, a padded batch
        dict(name="logp-shards-odd", op="logp", rows=12501, cols=1001, n=601, table="f32", x="bf16", ids="i32",
             scale=0.5, top=0, shards=2, pad=0.1),
        # a training micro-batch of 4096 tokens over the Llama-3-8B head
        dict(name="logp-batch", op="logp", rows=128256, cols=4096, n=4096, table="bf16", x="bf16", ids="i64",
             scale=1.0, top=0, shards=1, pad=0.0),
        # a short odd batch into a small fp32 table
        dict(name="grad-small", op="grad", rows=5003, cols=515, n=129, table="f32", x="f32", ids="i32", scale=1.0,
             pad=0.1, entropy=True, add=False),
        # 1024 tokens of GPT-2-small, added to the tied table's gradient
        dict(name="grad-tied", op="grad", rows=50257, cols=768, n=1024, table="bf16", x="bf16", ids="i64", scale=1.0,
             pad=0.0, entropy=False, add=True),
        # the micro-batch over the Llama-3-8B head, with an entropy bonus
        dict(name="grad-batch", op="grad", rows=128256, cols=4096, n=4096, table="bf16", x="bf16", ids="i64",
             scale=1.0, pad=0.02, entropy=True, add=False),
        # the smallest step: one matrix of an adapter
        dict(name="step8-small", op="step8", table="f32:96x160"),
        # the embeddings and biases of a small model, odd shapes and ragged groups
        dict(name="step8-ragged", op="step8", table="f32:50257x768,1024x768,1001*3"),
        # the owner of Llama-3-8B's embedding table (128256 x 4096 bf16, on AdamW)
        dict(name="step8-embedding-8b", op="step8", table="bf16:128256x4096"),
        # a run that goes over to 8 bits: one matrix, and GPT-2-small's table
        dict(name="moments-matrix", op="moments", table="f32:777x1001"),
        dict(name="moments-table", op="moments", table="f32:50257x768"),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logp", "logp", "grad", "grad", "step8", "moments"])
    if op in ("step8", "moments"):
        dt = rng.choice(["bf16", "f32"]) if op == "step8" else "f32"
        left, items = _between(rng, 2000, 300_000_000 if op == "step8" else 40_000_000), []
        while left > 0 and len(items) < (4 if op == "step8" else 1):
            rows = _between(rng, 1, 60000)
            cols = max(1, min(_between(rng, 1, 8192), left // rows))
            rows = min(rows, left)
            items.append("%dx%d" % (rows, cols))
            left -= rows * cols
        return dict(op=op, table="%s:%s" % (dt, ",".join(items)))
    rows, cols = _between(rng, 200, 130_000), _between(rng, 16, 4096)
    if rng.random() < 0.6:
        cols = (cols + 63) // 64 * 64
    table, x = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
    most = 4096 * 128256 * 4096 // (1 if table == x == "bf16" else 64)
    rows = min(rows, 200_000_000 // cols)
    case = dict(op=op, rows=rows, cols=cols, n=max(1, min(_between(rng, 1, 4096), most // (rows * cols))), table=table,
                x=x, ids=rng.choice(["i32", "i64"]), scale=rng.choice([1.0, 0.5, 1.4]), pad=rng.choice([0.0, 0.0, 0.1, 0.5]))
    if op == "logp":
        case.update(top=rng.choice([0, 1, 5, 20]) if case["n"] <= 512 else 0, shards=rng.choice([1, 1, 2]))
    else:
        case.update(entropy=rng.random() < 0.5, add=rng.random() < 0.4)
    return case


# ---- inputs ----

def _random(shape, scale, gen, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda").mul_(scale).to(dtype)


def _up(x, a):
    return -(-x // a) * a


def _shards(case):
    """[(first id, rows)] of the table's tensors."""
    s = case.get("shards", 1)
    cut = [case["rows"] * k // s for k in range(s + 1)]
    return list(zip(cut, np.diff(cut).tolist()))


def _hparams(B):
    return B.make_hparams(adam_lr=ADAM["lr"], adam_beta1=ADAM["beta1"], adam_beta2=ADAM["beta2"], adam_eps=ADAM["eps"],
                          adam_weight_decay=ADAM["weight_decay"])


def _space(nbytes):
    return torch.empty(max(nbytes, ALIGN), dtype=torch.uint8, device="cuda")


def _prepare_head(case, gen, s):
    n, rows, cols = case["n"], case["rows"], case["cols"]
    dt, xt = DTYPES[case["table"]], DTYPES[case["x"]]
    # the owner's flat buffer: a gain vector, then the table's tensors
    at, offs = 512, []
    for _, r in _shards(case):
        offs.append(at)
        at += _up(r * cols * dt.itemsize, ALIGN)
    s["buffer"] = torch.zeros(at, dtype=torch.uint8, device="cuda")
    s["weights"] = [s["buffer"][o:o + r * cols * dt.itemsize].view(dt).view(r, cols) for o, (_, r) in zip(offs, _shards(case))]
    # logits with a spread of about 3, as a model's
    if case.get("top"):
        # hidden states and weights on coarse grids (an 8-bit checkpoint): every fp32 sum is exact, so ranks are decided
        # and equal logits are really equal
        hidden = torch.randn(n, cols, generator=gen, device="cuda").mul_(2).round_().mul_(0.5)
        for w in s["weights"]:
            w.copy_(torch.randn(w.shape, generator=gen, device="cuda").mul_(16).round_().mul_(2.0 ** round(math.log2(3 / 16 / math.sqrt(cols)))))
    else:
        hidden = torch.randn(n, cols, generator=gen, device="cuda")
        for w in s["weights"]:
            w.copy_(_random(w.shape, 3 / math.sqrt(cols), gen))
    s["x"] = hidden.to(xt)
    # token ids of text: the frequency of a rank falls as its inverse; padding is negative
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    ids = torch.exp(u * math.log(rows + 1)).long().sub_(1).clamp_(0, rows - 1)
    padded = torch.rand(n, generator=gen, device="cuda") < case["pad"]
    s["ids"] = torch.where(padded, -100, ids).to(DTYPES[case["ids"]])
    if own:
        from matrix_optimizer_owner_amd import binding as B

        kind = B.BF16 if case["table"] == "bf16" else B.F32
        entries = [B.TableEntry(0, 1, 100, B.F32, B.ROLE_ADAMW)]
        entries += [B.TableEntry(o, r, cols, kind, B.ROLE_ADAMW8) for o, (_, r) in zip(offs, _shards(case))]
        s["plan"] = B.OwnerPlan(entries, at, _hparams(B))
        s["call"] = dict(id_type=B.I64 if case["ids"] == "i64" else B.I32, x_type=B.BF16 if case["x"] == "bf16" else B.F32,
                         scale=case["scale"])
        s["total"] = B.head_total
        s["record"] = B.HEAD_RECORD_BYTES
        top = case.get("top", 0)
        need = max(s["plan"].head_workspace_bytes(1 + k, n, x_type=s["call"]["x_type"], top_k=top, grad=case["op"] == "grad")
                   for k in range(len(offs)))
        s["space"] = _space(need)
        s["records"] = _space(n * s["record"] * len(offs))
    if case["op"] == "logp":
        s["logp"] = torch.empty(n, device="cuda")
        s["entropy"] = torch.empty(n, device="cuda")
        k = case["top"]
        if k:
            s["top_ids"] = torch.empty(len(offs), n, k, dtype=torch.int64, device="cuda")
            s["top_logp"] = torch.empty(len(offs), n, k, device="cuda")
            s["all_ids"] = torch.empty(n, k, dtype=torch.int64, device="cuda") if len(offs) > 1 else s["top_ids"][0]
            s["all_logp"] = torch.empty(n, k, device="cuda") if len(offs) > 1 else s["top_logp"][0]
        return s
    s["dlogp"] = _random((n,), 0.3, gen).sub_(1.0).div_(n)  # a mean of -logp, each token with a weight
    s["dentropy"] = torch.full((n,), 0.05 / n, device="cuda") if case["entropy"] else None
    s["grads"] = torch.zeros_like(s["buffer"])
    g = s["dtable"] = s["grads"][offs[0]:offs[0] + rows * cols * dt.itemsize].view(dt).view(rows, cols)
    if case["add"]:
        g.copy_(_random(g.shape, 1e-4, gen))
    s["dx"] = torch.empty_like(s["x"])
    # what the forward pass left: the rows' log sum of exponentials and entropy, for the plain form and the framework
    # each in its own form
    if own:
        s["plan"].head_logprob(1, s["buffer"].data_ptr(), s["x"].data_ptr(), n, s["records"].data_ptr(), s["space"].data_ptr(),
                               s["space"].numel(), ids=s["ids"].data_ptr(),
                               stream=torch.cuda.current_stream().cuda_stream, **s["call"])
    else:
        s["lse"], s["entropy"] = _plain_stats(_plain_logits(s))
    return s


def _tensors(table):
    """(dtype, [(rows, cols)]) of a table text "dtype:ROWSxCOLS*COUNT,..."."""
    dt, items = table.split(":")
    out = []
    for item in items.split(","):
        shape, _, count = item.partition("*")
        r, _, c = shape.rpartition("x")
        out += [(int(r or 1), int(c))] * int(count or 1)
    return DTYPES[dt], out


def _quantised(m, r):
    """Codes and scales of whole groups (rows of m and r) of the first moment and of the second's root, to nearest."""
    sm, sr = m.abs().amax(1, keepdim=True), r.amax(1, keepdim=True)
    cm = torch.floor(127 * (m.abs() / sm.clamp_min(1e-30)).sqrt() + 0.5)
    cr = torch.floor(255 * (r / sr.clamp_min(1e-30)).sqrt() + 0.5)
    cr = torch.where(r > 0, cr.clamp_min(1), cr)
    return (cm * torch.sign(m)).to(torch.int8), sm, cr.to(torch.uint8), sr


def _prepare_state(case, gen, s):
    dt, shapes = _tensors(case["table"])
    numel = np.array([r * c for r, c in shapes])
    groups = -(-numel // GROUP)
    first = np.concatenate([[0], np.cumsum(groups)])  # first group of each tensor
    total = int(first[-1])
    s.update(dt=dt, total=total)
    # every tensor starts at a whole group: the flat buffer is rows of GROUP elements, the last of a tensor ragged
    valid = None
    if (numel % GROUP).any():
        held = torch.full((total,), GROUP, dtype=torch.int32)
        held[torch.from_numpy(first[1:] - 1)] = torch.from_numpy((numel - (groups - 1) * GROUP).astype(np.int32))
        valid = torch.arange(GROUP, device="cuda") < held.cuda()[:, None]
    s["valid"] = valid
    keep = 1.0 if valid is None else valid
    # the moments of a run: gradients of one size a group, averaged over some steps
    size = 10.0 ** (torch.rand(total, 1, generator=gen, device="cuda") * 2 - 4)
    m = _random((total, GROUP), 0.25, gen).mul_(size).mul_(keep)
    r = _random((total, GROUP), 0.2, gen).add_(1.0).abs_().clamp_(0.3).mul_(size).mul_(keep)
    if case["op"] == "moments":
        s["m"], s["v"] = m, r.square_()
    else:
        s["codes"] = list(_quantised(m, r))
        del m, r
        s["params"] = _random((total, GROUP), 0.02, gen, dt)
        g = _random((total, GROUP), 1.0, gen).mul_(size)
        # the bytes between two tensors belong to nobody and hold anything
        s["grads"] = (g if valid is None else torch.where(valid, g, math.nan)).to(dt)
        s["factor"] = torch.full((1,), 0.7, device="cuda") + 0.1 * torch.rand(1, generator=gen, device="cuda")
        s["step"] = 11
        # each group's tensor, and the group's place in it
        s["tensor"] = torch.repeat_interleave(torch.arange(len(groups)), torch.from_numpy(groups)).cuda()
        s["place"] = torch.arange(total, device="cuda") - torch.from_numpy(first[:-1]).cuda()[s["tensor"]]
    if own:
        from matrix_optimizer_owner_amd import binding as B

        entries = [B.TableEntry(int(f) * GROUP * dt.itemsize, r, c, B.BF16 if dt == torch.bfloat16 else B.F32, B.ROLE_ADAMW8)
                   for f, (r, c) in zip(first, shapes)]
        s["plan"] = B.OwnerPlan(entries, total * GROUP * dt.itemsize, _hparams(B))
        s["state"] = torch.zeros(s["plan"].state_bytes, dtype=torch.uint8, device="cuda")
        s["starts"] = [int(f) * GROUP for f in first[:-1]]
        s["F32"], s["BF16"] = B.F32, B.BF16
        s["m_out"] = torch.zeros(total, GROUP, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros_like(s["m_out"])
        if case["op"] == "step8":
            cm, sm, cr, sr = s.pop("codes")
            for i, k in enumerate(numel):
                info, a, b = s["plan"].entry_info(i), int(first[i]), int(first[i + 1])
                for off, code, scale in ((info.state_offset, cm, sm), (info.state_offset2, cr, sr)):
                    s["state"][off:off + (b - a) * GROUP].copy_(code[a:b].view(torch.uint8).view(-1))
                    off += _up(int(k), ALIGN)
                    s["state"][off:off + 4 * (b - a)].view(torch.float32).copy_(scale[a:b, 0])
            s["space"] = _space(s["plan"].workspace_bytes)
            s["flags"], s["resident"] = 0, B.STEP_DESCRIPTORS_RESIDENT
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    return _prepare_head(case, gen, s) if case["op"] in ("logp", "grad") else _prepare_state(case, gen, s)


# ---- one pass, plain ----

def _plain_logits(s):
    w = s["weights"][0] if len(s["weights"]) == 1 else torch.cat(s["weights"])
    return (s["x"].float() @ w.float().t()).mul_(s["case"]["scale"])


def _plain_stats(z):
    most = z.amax(1, keepdim=True)
    e = torch.exp(z - most)
    total = e.sum(1, keepdim=True)
    entropy = total.log() - (e * (z - most)).sum(1, keepdim=True) / total
    return (most + total.log())[:, 0], entropy[:, 0]


def _plain_logp(s):
    z = _plain_logits(s)
    lse, entropy = _plain_stats(z)
    ids = s["ids"].long()
    here = ids >= 0
    logp = z.gather(1, ids.clamp_min(0)[:, None])[:, 0] - lse
    out = [torch.where(here, logp, 0.0), torch.where(here, entropy, 0.0)]
    k = s["case"]["top"]
    if k:
        top, at = torch.sort(z, dim=1, descending=True, stable=True)
        out += [torch.where(here[:, None], at[:, :k], -1), torch.where(here[:, None], top[:, :k] - lse[:, None], -math.inf)]
    return out


def _plain_grad(s):
    case, ids = s["case"], s["ids"].long()
    here = ids >= 0
    logp = _plain_logits(s).sub_(s["lse"][:, None])
    p = logp.exp()
    dlogp = torch.where(here, s["dlogp"], 0.0)
    dz = p * -dlogp[:, None]
    if case["entropy"]:
        dz -= torch.where(here, s["dentropy"], 0.0)[:, None] * p * (logp + s["entropy"][:, None])
    dz.scatter_add_(1, ids.clamp_min(0)[:, None], dlogp[:, None])
    dz *= case["scale"]
    s["dx"].copy_(dz @ s["weights"][0].float())
    dw = dz.t() @ s["x"].float()
    s["dtable"].copy_(dw.add_(s["dtable"].float()) if case["add"] else dw)
    return [s["dx"], s["dtable"]]


_WORD = 0xFFFFFFFF


def _mix(h):
    """The finaliser of MurmurHash3 on 32-bit words held in int64."""
    h = (h ^ (h >> 16)) * 0x85EBCA6B & _WORD
    h = (h ^ (h >> 13)) * 0xC2B2AE35 & _WORD
    return h ^ (h >> 16)


def _dither(s):
    """What is added before a code is rounded down, for the first moment and the second's root: in (0, 1), from step, tensor
    and element; a 32-bit word for two elements, a byte for each value."""
    key = _mix((s["step"] + 0x9E3779B9 * (s["tensor"] + 1)) & _WORD)
    pair = s["place"][:, None] * (GROUP // 2) + torch.arange(GROUP // 2, device="cuda")
    word = _mix((pair + key[:, None]) & _WORD)
    parts = torch.stack([word >> k & 0xFF for k in (0, 16, 8, 24)], 2).float().add_(0.5).mul_(1 / 256)
    return parts[:, :, :2].reshape(-1, GROUP), parts[:, :, 2:].reshape(-1, GROUP)


def _plain_step(s):
    cm, sm, cr, sr = s["codes"]
    a = ADAM
    g = s["grads"].float() * s["factor"]
    if s["valid"] is not None:
        g = torch.where(s["valid"], g, 0.0)
    c = cm.float()
    m = a["beta1"] * (c * c.abs() * (sm / 16129)) + (1 - a["beta1"]) * g
    r = cr.float().square() * (sr / 65025)
    v = a["beta2"] * r * r + (1 - a["beta2"]) * g * g
    w = s["params"].float()
    new = w * (1 - a["lr"] * a["weight_decay"]) - a["lr"] * (m / (1 - a["beta1"] ** s["step"])) / (
        (v / (1 - a["beta2"] ** s["step"])).sqrt() + a["eps"])
    s["params"].copy_(new if s["valid"] is None else torch.where(s["valid"], new, w))
    um, ur = _dither(s)
    r = v.sqrt()
    sm, sr = m.abs().amax(1, keepdim=True), r.amax(1, keepdim=True)
    c = torch.floor(127 * (m.abs() / sm.clamp_min(1e-30)).sqrt() + um).clamp_max(127) * torch.sign(m)
    d = torch.floor(255 * (r / sr.clamp_min(1e-30)).sqrt() + ur).clamp_max(255)
    d = torch.where(r > 0, d.clamp_min(1), 0.0)
    s["codes"] = [c.to(torch.int8), sm, d.to(torch.uint8), sr]
    # what is held in 8 bits, as the values it stands for
    return [s["params"], (c * c.abs() * (sm / 16129)).bfloat16(), (d * d * (sr / 65025)).square().bfloat16()]


def _plain_moments(s):
    cm, sm, cr, sr = _quantised(s["m"], s["v"].sqrt())
    c, d = cm.float(), cr.float()
    return [(c * c.abs() * (sm / 16129)).bfloat16(), (d * d * (sr / 65025)).square().bfloat16()]


# ---- one pass, the framework's ----

def _own_logp(s, stream):
    case, plan, n, k = s["case"], s["plan"], s["case"]["n"], s["case"]["top"]
    parts = _shards(case)
    alone = len(parts) == 1
    records = s["records"].data_ptr()
    for i, (first, _) in enumerate(parts):
        plan.head_logprob(1 + i, s["buffer"].data_ptr(), s["x"].data_ptr(), n, records + i * n * s["record"],
                          s["space"].data_ptr(), s["space"].numel(), ids=s["ids"].data_ptr(), first_id=first,
                          logp=s["logp"].data_ptr() if alone else 0, entropy=s["entropy"].data_ptr() if alone else 0,
                          top_k=k, top_ids=s["top_ids"][i].data_ptr() if k else 0,
                          top_logp=s["top_logp"][i].data_ptr() if k and alone else 0,
                          top_logits=s["top_logp"][i].data_ptr() if k and not alone else 0, stream=stream, **s["call"])
    if not alone:
        s["total"](records, len(parts), n, records, logp=s["logp"].data_ptr(), entropy=s["entropy"].data_ptr(), top_k=k,
                   part_top_ids=s["top_ids"].data_ptr() if k else 0, part_top_logits=s["top_logp"].data_ptr() if k else 0,
                   top_ids=s["all_ids"].data_ptr() if k else 0, top_logp=s["all_logp"].data_ptr() if k else 0, stream=stream)
    return [s["logp"], s["entropy"]] + ([s["all_ids"], s["all_logp"]] if k else [])


def _own(s):
    case, plan = s["case"], s["plan"]
    op = case["op"]
    stream = torch.cuda.current_stream().cuda_stream
    if op == "logp":
        return _own_logp(s, stream)
    if op == "grad":
        plan.head_grad(1, s["buffer"].data_ptr(), s["grads"].data_ptr(), s["x"].data_ptr(), case["n"],
                       s["records"].data_ptr(), s["dlogp"].data_ptr(), s["space"].data_ptr(), s["space"].numel(),
                       dentropy=s["dentropy"].data_ptr() if case["entropy"] else 0, dx=s["dx"].data_ptr(),
                       ids=s["ids"].data_ptr(), accumulate=case["add"], stream=stream, **s["call"])
        return [s["dx"], s["dtable"]]
    state = s["state"].data_ptr()
    if op == "step8":
        plan.step_scaled(s["params"].data_ptr(), s["grads"].data_ptr(), state, s["space"].data_ptr(), s["space"].numel(),
                         s["step"], s["factor"].data_ptr(), stream=stream, flags=s["flags"])
        s["flags"] = s["resident"]  # the workspace holds the plan's descriptors from the first pass on
    else:
        plan.moments_write(0, state, s["m"].data_ptr(), s["v"].data_ptr(), type=s["F32"], stream=stream)
    for i, at in enumerate(s["starts"]):
        plan.moments_read(i, state, s["m_out"].data_ptr() + 2 * at, s["v_out"].data_ptr() + 2 * at, type=s["BF16"],
                          stream=stream)
    return ([s["params"]] if op == "step8" else []) + [s["m_out"], s["v_out"]]


def run(state):
    if own:
        return _own(state)
    return {"logp": _plain_logp, "grad": _plain_grad, "step8": _plain_step, "moments": _plain_moments}[state["case"]["op"]](state)


# ---- what one pass cannot do without ----

def work(case):
    if case["op"] in ("logp", "grad"):
        n, rows, cols = case["n"], case["rows"], case["cols"]
        es, ex = DTYPES[case["table"]].itemsize, DTYPES[case["x"]].itemsize
        read = rows * cols * es + n * (cols * ex + DTYPES[case["ids"]].itemsize)
        if case["op"] == "logp":
            return {"bytes": read + n * (8 + 12 * case["top"]), "flops": 2 * n * rows * cols}
        # logits again from the rows' sums, then the two products
        return {"bytes": read + n * (cols * ex + 20) + (2 if case["add"] else 1) * rows * cols * es, "flops": 6 * n * rows * cols}
    dt, shapes = _tensors(case["table"])
    numel = sum(r * c for r, c in shapes)
    scales = 8 * sum(-(-r * c // GROUP) for r, c in shapes)
    if case["op"] == "step8":  # parameters and two codes read and written, gradients read; the values read out of the codes
        return {"bytes": numel * (3 * dt.itemsize + 4 + 2 + 4) + 3 * scales, "flops": 40 * numel}
    return {"bytes": numel * (8 + 2 + 2 + 4) + 2 * scales, "flops": 20 * numel}


# ---- the definition in 64 bits ----

def _exact_head(case, s):
    n, k = case["n"], case.get("top", 0)
    x, w = s["x"].double(), torch.cat(s["weights"]).double()
    ids = s["ids"].cpu().numpy().astype(np.int64)
    outs = [np.zeros(n), np.zeros(n), np.full((n, max(k, 1)), -1, dtype=np.int64), np.full((n, max(k, 1)), -np.inf)]
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    for a in range(0, n, 512):
        rows = np.arange(a, min(n, a + 512))
        live = rows[ids[rows] >= 0]
        if not len(live):
            continue
        at = torch.from_numpy(live).cuda()
        target = torch.from_numpy(ids[live]).cuda()
        logp = torch.log_softmax(torch.matmul(x[at], w.T) * case["scale"], 1)
        p = torch.exp(logp)
        entropy = -(p * logp).sum(1)
        line = torch.arange(len(live), device="cuda")
        outs[0][live] = logp[line, target].cpu().numpy()
        outs[1][live] = entropy.cpu().numpy()
        if k:
            order = np.lexsort((np.broadcast_to(np.arange(case["rows"]), p.shape), -logp.cpu().numpy()), axis=1)[:, :k] \
                if case["rows"] * len(live) <= 20_000_000 else None
            if order is None:
                return None
            outs[2][live] = order
            outs[3][live] = np.take_along_axis(logp.cpu().numpy(), order, 1)
        if case["op"] == "grad":
            one = torch.zeros_like(p)
            one[line, target] = 1.0
            dz = (one - p) * s["dlogp"].double()[at][:, None]
            if case["entropy"]:
                dz = dz - p * (logp + entropy[:, None]) * s["dentropy"].double()[at][:, None]
            dz = dz * case["scale"]
            dx[at] = torch.matmul(dz, w)
            dw += torch.matmul(dz.T, x[at])
    if case["op"] == "logp":
        return outs if k else outs[:2]
    return [dx, dw + s["dtable"].double() if case["add"] else dw]


def _exact_codes(value, most, count, shift, least):
    """|value| / most as squares of whole numbers below `count`, rounded down after `shift`."""
    share = torch.where(most > 0, value.abs() / most, 0.0)
    code = torch.clamp(torch.floor(torch.sqrt(share) * count + shift), max=count)
    return torch.where((value != 0) & (code < least), float(least), code)


def _exact_state(case, s):
    dt, shapes = _tensors(case["table"])
    outs = [[], [], []]
    at = 0
    for t, (rows, cols) in enumerate(shapes):
        k = rows * cols
        groups = -(-k // GROUP)
        cut = slice(at, at + groups)
        at += groups
        flat = lambda v: v[cut].reshape(-1)[:k].double()  # noqa: E731
        over = lambda v: torch.nn.functional.pad(v, (0, groups * GROUP - k)).view(groups, GROUP)  # noqa: E731
        if case["op"] == "moments":
            m, v = flat(s["m"]), flat(s["v"])
            um = ur = 0.5
        else:
            cm, sm, cr, sr = s["codes"]
            wide = lambda v: v[cut].double().expand(-1, GROUP).reshape(-1)[:k]  # noqa: E731
            g = flat(s["grads"]) * float(s["factor"])
            m = ADAM["beta1"] * wide(sm) * torch.sign(flat(cm)) * (flat(cm) / 127) ** 2 + (1 - ADAM["beta1"]) * g
            v = ADAM["beta2"] * (wide(sr) * (flat(cr) / 255) ** 2) ** 2 + (1 - ADAM["beta2"]) * g ** 2
            w = flat(s["params"])
            move = m / (1 - ADAM["beta1"] ** s["step"]) / (torch.sqrt(v / (1 - ADAM["beta2"] ** s["step"])) + ADAM["eps"])
            w = w - ADAM["lr"] * (ADAM["weight_decay"] * w + move)
            whole = s["params"][cut].double().reshape(-1)
            whole[:k] = w
            outs[0].append(whole.view(groups, GROUP))

            def hashed(h):
                h = h ^ h >> np.uint32(16)
                h = h * np.uint32(0x85EBCA6B)
                h = h ^ h >> np.uint32(13)
                h = h * np.uint32(0xC2B2AE35)
                return h ^ h >> np.uint32(16)

            key = hashed(np.array([(s["step"] + 0x9E3779B9 * (t + 1)) % 2 ** 32], dtype=np.uint32))
            part = hashed(np.arange(groups * GROUP // 2, dtype=np.uint32) + key).view(np.uint8).reshape(-1, 2, 2)
            um, ur = (torch.from_numpy(np.ascontiguousarray(part[:, :, j]).reshape(groups, GROUP)).cuda().double() / 256 + 1 / 512
                      for j in (0, 1))
        m, r = over(m), over(torch.sqrt(v))
        sm, sr = m.abs().amax(1, keepdim=True), r.amax(1, keepdim=True)
        outs[1].append(sm * (_exact_codes(m, sm, 127, um, 0) / 127) ** 2 * torch.sign(m))
        outs[2].append((sr * (_exact_codes(r, sr, 255, ur, 1) / 255) ** 2) ** 2)
    return [torch.cat(o) for o in outs if o]


def exact(case, seed):
    global own
    mine, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = mine
    return _exact_head(case, s) if case["op"] in ("logp", "grad") else _exact_state(case, s)
