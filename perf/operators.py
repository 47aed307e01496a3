"""Cases of the operators around the owner step: what the gradients of a flat
owner buffer go through before the optimizer reads them, and an embedding
table that lives in that buffer.

Operators (field "op" of a case):

  norm    the global L2 norm of every gradient of the buffer, the norm of each
          tensor, and the factor min(1, max_norm / (norm + eps));
  clip    norm, then every gradient times that factor, into a second buffer;
  step    norm, then the AdamW step with that factor applied to the gradients
          as they are read;
  lookup  out[i] = scale * table[token[i] - first], a zero row for an id
          outside the table;
  embed   the table's gradient, grad[v] (+)= scale * sum of dout[i] over the
          positions i with token[i] - first = v.

``run`` computes a case in plain torch operations, or through the package
where ``own`` is true.  ``exact`` computes it in 64 bits from the definition.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "i32": torch.int32, "i64": torch.int64}
ADAM = dict(lr=0.02, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.01)
EPS = 1e-6
ALIGN = 256


def listed():
    return [
        # the norm gains of a 32-layer model, the smallest tail an owner holds: launch latency
        dict(name="norm-gains", op="norm", table="f32:4096*65", max_norm=0.1),
        # one owner's share of Llama-3-8B: 28 matrices, 872 M gradients in bf16
        dict(name="norm-share-8b", op="norm",
             table="bf16:4096x4096*8,1024x4096*8,14336x4096*8,4096x14336*4", max_norm=1.0),
        # a small model with odd shapes: bf16 matrices, fp32 biases, ragged ends everywhere
        dict(name="clip-ragged", op="clip", table="bf16:777x1001*4,520x130*6,33x45*12,1x1;f32:333*40,77x5*8",
             max_norm=0.5),
        # the Llama-3-8B share clipped before a step that keeps the raw gradients
        dict(name="clip-share-8b", op="clip",
             table="bf16:4096x4096*8,1024x4096*8,14336x4096*8,4096x14336*4", max_norm=1.0),
        # a tail owner's clipped step over the gains and biases of a small model
        dict(name="step-tail", op="step", table="f32:768*50,2304*24,1001*3", max_norm=0.1),
        # the owner of Llama-3-8B's embedding table (128256 x 4096 bf16, on AdamW)
        dict(name="step-embedding-8b", op="step", table="bf16:128256x4096", max_norm=1.0),
        # token ids of one decoding step of 32 sequences, scaled by sqrt(width)
        dict(name="lookup-decode", op="lookup", rows=128256, cols=4096, tokens=32, first=0, table="bf16",
             out="bf16", ids="i64", scale=64.0, outside=0.0),
        # a training micro-batch of 4 x 4096 tokens
        dict(name="lookup-batch", op="lookup", rows=128256, cols=4096, tokens=16384, first=0, table="bf16",
             out="bf16", ids="i64", scale=1.0, outside=0.0),
        # a vocabulary shard with an odd width: fp32 table, bf16 activations, ids of other shards
        dict(name="lookup-shard-odd", op="lookup", rows=12501, cols=1001, tokens=6001, first=12501, table="f32",
             out="bf16", ids="i32", scale=0.5, outside=0.5),
        # a short odd batch into a small table
        dict(name="embed-small", op="embed", rows=5003, cols=515, tokens=129, first=0, table="f32", out="f32",
             ids="i32", scale=1.0, outside=0.1, add=False),
        # the micro-batch's gradient of the whole Llama-3-8B table
        dict(name="embed-batch", op="embed", rows=128256, cols=4096, tokens=16384, first=0, table="bf16",
             out="bf16", ids="i64", scale=1.0, outside=0.0, add=False),
        # a 64 x 1024 batch added to the tied output head's gradient, GPT-2-small's width
        dict(name="embed-tied", op="embed", rows=50257, cols=768, tokens=65536, first=0, table="f32", out="bf16",
             ids="i64", scale=1.0, outside=0.02, add=True),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "clip", "step", "lookup", "embed", "embed"])
    if op in ("norm", "clip"):
        left, parts = _between(rng, 4000, 200_000_000), {"bf16": [], "f32": []}
        kind = rng.choice(["bf16", "f32", "both"])
        while left > 0 and len(parts["bf16"]) + len(parts["f32"]) < 60:
            rows, cols = _between(rng, 1, 8192), _between(rng, 1, 16384)
            count = max(1, min(rng.randint(1, 12), left // (rows * cols) if rows * cols <= left else 1))
            if rows * cols > left:
                rows = max(1, left // cols)
            parts[rng.choice(["bf16", "f32"]) if kind == "both" else kind].append("%dx%d*%d" % (rows, cols, count))
            left -= rows * cols * count
        table = ";".join("%s:%s" % (d, ",".join(p)) for d, p in parts.items() if p)
        return dict(op=op, table=table, max_norm=rng.choice([0.01, 0.1, 1.0, 1000.0]))
    if op == "step":
        if rng.random() < 0.5:
            table = "bf16:%dx%d" % (_between(rng, 64, 60000), 128 * rng.randint(1, 40))
        else:
            table = "f32:" + ",".join("%d*%d" % (_between(rng, 1, 500_000), rng.randint(1, 30)) for _ in range(rng.randint(1, 6)))
        return dict(op=op, table=table, max_norm=rng.choice([0.01, 0.1, 1.0, 1000.0]))
    rows, cols = _between(rng, 100, 200_000), _between(rng, 8, 8192)
    if rng.random() < 0.5:
        cols = (cols + 7) // 8 * 8
    rows = min(rows, 400_000_000 // cols)
    tokens = min(_between(rng, 1, 65536), 200_000_000 // cols)
    case = dict(op=op, rows=rows, cols=cols, tokens=tokens, first=rng.choice([0, 0, rows]),
                table=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]), ids=rng.choice(["i32", "i64"]),
                scale=rng.choice([1.0, 0.5, 22.6]), outside=rng.choice([0.0, 0.0, 0.1, 0.5]))
    if op == "embed":
        case["add"] = rng.random() < 0.4
    return case


# ---- the flat buffer of a table of tensors ----

def _tensors(table):
    """[(dtype, rows, cols)] of a table text: "dtype:ROWSxCOLS*COUNT,...;dtype:..." (bf16 tensors first)."""
    out = []
    for group in table.split(";"):
        dt, items = group.split(":")
        for item in items.split(","):
            shape, _, count = item.partition("*")
            r, _, c = shape.rpartition("x")
            out += [(dt, int(r or 1), int(c))] * int(count or 1)
    return out


def _layout(tensors):
    """Byte offsets (256-byte aligned) and the size of the flat buffer."""
    offs, at = [], 0
    for dt, r, c in tensors:
        offs.append(at)
        at += -(-r * c * DTYPES[dt].itemsize // ALIGN) * ALIGN
    return offs, at


def _groups(tensors, offs, nbytes, device):
    """Per dtype the contiguous run of the buffer that holds it, as rows of 256 bytes: (dtype, first byte, last
    byte, which elements are a tensor's own (None: all of them), last row of each tensor, tensors before it)."""
    got = []
    for name in ("bf16", "f32"):
        mine = [i for i, t in enumerate(tensors) if t[0] == name]
        if not mine:
            continue
        per = ALIGN // DTYPES[name].itemsize
        lo = offs[mine[0]]
        numel = np.array([tensors[i][1] * tensors[i][2] for i in mine])
        rows = -(-numel // per)
        ends = np.cumsum(rows)
        hi = lo + int(ends[-1]) * ALIGN
        mask = None
        if (numel % per).any():
            valid = torch.full((int(ends[-1]),), per, dtype=torch.int32)
            valid[torch.from_numpy(ends - 1)] = torch.from_numpy((numel - (rows - 1) * per).astype(np.int32))
            mask = torch.arange(per, device=device) < valid.to(device)[:, None]
        got.append((DTYPES[name], lo, hi, mask, torch.from_numpy(ends - 1).to(device), mine[0], rows))
    return got


def _random(shape, scale, gen, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda").mul_(scale).to(dtype)


def _zipf(case, gen):
    """Token ids of text: the frequency of a rank falls as its inverse; a share of them outside the table."""
    n, rows = case["tokens"], case["rows"]
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    ids = torch.exp(u * math.log(rows + 1)).long().sub_(1).clamp_(0, rows - 1) + case["first"]
    if case["outside"]:
        away = torch.rand(n, generator=gen, device="cuda") < case["outside"]
        ids = torch.where(away, torch.where(u < 0.5, ids + rows, ids - rows - case["first"] - 1), ids)
    return ids.to(DTYPES[case["ids"]])


def _plan(tensors, offs, nbytes):
    from matrix_optimizer_owner_amd import binding as B

    entries = [B.TableEntry(o, r, c, B.BF16 if d == "bf16" else B.F32, B.ROLE_ADAMW) for o, (d, r, c) in zip(offs, tensors)]
    hp = B.make_hparams(adam_lr=ADAM["lr"], adam_beta1=ADAM["beta1"], adam_beta2=ADAM["beta2"], adam_eps=ADAM["eps"],
                        adam_weight_decay=ADAM["weight_decay"])
    return B, B.OwnerPlan(entries, nbytes, hp)


def _space(nbytes):
    return torch.empty(max(nbytes, ALIGN), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    if case["op"] in ("lookup", "embed"):
        # a gain vector, then the table: one owner's flat buffer
        tensors = [("f32", 1, 100), (case["table"], case["rows"], case["cols"])]
        offs, nbytes = _layout(tensors)
        s["buffer"] = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
        span = case["rows"] * case["cols"] * DTYPES[case["table"]].itemsize
        s["weight"] = s["buffer"][offs[1]:offs[1] + span].view(DTYPES[case["table"]]).view(case["rows"], case["cols"])
        s["weight"].copy_(_random(s["weight"].shape, 0.02, gen))
        s["ids"] = _zipf(case, gen)
        shape = (case["tokens"], case["cols"])
        if case["op"] == "lookup":
            s["out"] = torch.empty(shape, dtype=DTYPES[case["out"]], device="cuda")
        else:
            s["dout"] = _random(shape, 0.01, gen, DTYPES[case["out"]])
        if own:
            B, s["plan"] = _plan(tensors, offs, nbytes)
            s["out_type"] = B.BF16 if case["out"] == "bf16" else B.F32
            s["id_type"] = B.I64 if case["ids"] == "i64" else B.I32
            if case["op"] == "embed":
                s["space"] = _space(s["plan"].embed_workspace_bytes(1, case["tokens"]))
        return s
    tensors = _tensors(case["table"])
    offs, nbytes = _layout(tensors)
    s.update(tensors=tensors, groups=_groups(tensors, offs, nbytes, "cuda"), n=len(tensors))
    s["grads"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    std = 10.0 ** (torch.rand(s["n"], generator=gen, device="cuda") * 2 - 4)  # each tensor at a scale of its own
    for dt, lo, hi, mask, last, first, rows in s["groups"]:
        which = torch.repeat_interleave(torch.arange(len(rows)), torch.from_numpy(rows)).cuda() + first
        v = _random((len(which), ALIGN // dt.itemsize), 1.0, gen).mul_(std[which][:, None])
        # the bytes between two tensors belong to nobody and hold anything
        s["grads"][lo:hi].view(dt).view(v.shape).copy_(v if mask is None else torch.where(mask, v, math.nan))
    s["stats"] = torch.zeros(4, dtype=torch.float32, device="cuda")
    if case["op"] == "norm":
        s["norms"] = torch.empty(s["n"], dtype=torch.float32, device="cuda")
    if case["op"] == "clip":
        s["out"] = torch.zeros_like(s["grads"])
    if case["op"] == "step":
        numel = [r * c for _, r, c in tensors]
        cells = np.array([-(-k * 4 // ALIGN) for k in numel])  # moments: fp32, m then v of each tensor, 256-byte aligned
        s["params"] = torch.zeros_like(s["grads"])
        dt, lo, hi, mask, last, first, rows = s["groups"][0]
        w = s["params"].view(dt)
        w.copy_(_random(w.shape, 0.02, gen))
        at = np.concatenate([[0], np.cumsum(2 * cells)[:-1]])
        m_cells = np.concatenate([a + np.arange(k) for a, k in zip(at, cells)])
        v_cells = np.concatenate([a + k + np.arange(k) for a, k in zip(at, cells)])
        whole = len(tensors) == 1  # one tensor: a plain range of the state
        s["m_at"] = slice(0, int(cells[0])) if whole else torch.from_numpy(m_cells).cuda()
        s["v_at"] = slice(int(cells[0]), int(2 * cells[0])) if whole else torch.from_numpy(v_cells).cuda()
        s["state"] = torch.zeros(int(2 * cells.sum()) * 64, dtype=torch.float32, device="cuda")
        keep = torch.ones(1, device="cuda") if mask is None else mask.view(-1, 64)
        cell = s["state"].view(-1, 64)
        cell[s["m_at"]] = _random((len(m_cells), 64), 1e-3, gen) * keep
        cell[s["v_at"]] = _random((len(v_cells), 64), 1e-3, gen).square_() * keep
        s["step"] = 11
    if own:
        B, s["plan"] = _plan(tensors, offs, nbytes)
        s["space"] = _space(s["plan"].grad_workspace_bytes)
        s["step_space"] = _space(s["plan"].workspace_bytes) if case["op"] == "step" else None
        s["flags"] = 0
        s["resident"] = B.STEP_DESCRIPTORS_RESIDENT
    return s


# ---- one pass ----

def _plain_norm(s, max_norm):
    """(norm of each tensor, [norm, factor]) with sums of a row in 32 bits and the long sums in 64."""
    parts = []
    for dt, lo, hi, mask, last, first, rows in s["groups"]:
        x = s["grads"][lo:hi].view(dt).view(-1, ALIGN // dt.itemsize).float()
        if mask is not None:
            x = torch.where(mask, x, 0.0)
        run_ = (x * x).sum(1).double().cumsum(0)[last]
        parts.append(torch.diff(run_, prepend=run_.new_zeros(1)))
    sums = torch.cat(parts)
    norm = sums.sum().sqrt()
    factor = (max_norm / (norm + EPS)).clamp(max=1.0)
    return sums.sqrt().float(), torch.stack([norm, factor]).float()


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "lookup":
        at = s["ids"].long() - case["first"]
        inside = (at >= 0) & (at < case["rows"])
        w = s["weight"][at.clamp(0, case["rows"] - 1)].float() * case["scale"]
        return torch.where(inside[:, None], w, 0.0).to(DTYPES[case["out"]])
    if op == "embed":
        at = s["ids"].long() - case["first"]
        at = torch.where((at >= 0) & (at < case["rows"]), at, case["rows"])
        acc = torch.zeros(case["rows"] + 1, case["cols"], device="cuda").index_add_(0, at, s["dout"].float())
        acc = acc[:-1].mul_(case["scale"])
        s["weight"].copy_(acc.add_(s["weight"].float()) if case["add"] else acc)
        return s["weight"]
    norms, stats = _plain_norm(s, case["max_norm"])
    if op == "norm":
        return [norms, stats]
    factor = stats[1]
    if op == "clip":
        outs = [(s["out"][lo:hi].view(dt), s["grads"][lo:hi].view(dt), mask) for dt, lo, hi, mask, *_ in s["groups"]]
        done = [o.copy_(g.float() * factor) if m is None else o.copy_(torch.where(m.view(-1), g.float() * factor, 0.0)) for o, g, m in outs]
        return [stats] + done
    dt, lo, hi, mask, *_ = s["groups"][0]
    g = s["grads"].view(dt).float() * factor
    w = s["params"].view(dt).float()
    if mask is not None:
        g = torch.where(mask.view(-1), g, 0.0)
    cell = s["state"].view(-1, 64)
    m = ADAM["beta1"] * cell[s["m_at"]].view(-1) + (1 - ADAM["beta1"]) * g
    v = ADAM["beta2"] * cell[s["v_at"]].view(-1) + (1 - ADAM["beta2"]) * g * g
    mh = m / (1 - ADAM["beta1"] ** s["step"])
    vh = v / (1 - ADAM["beta2"] ** s["step"])
    new = w * (1 - ADAM["lr"] * ADAM["weight_decay"]) - ADAM["lr"] * mh / (vh.sqrt() + ADAM["eps"])
    s["params"].view(dt).copy_(new if mask is None else torch.where(mask.view(-1), new, w))
    cell[s["m_at"]] = m.view(-1, 64)
    cell[s["v_at"]] = v.view(-1, 64)
    return [stats, s["params"].view(dt), s["state"]]


def _own(s):
    case, plan = s["case"], s["plan"]
    op = case["op"]
    stream = torch.cuda.current_stream().cuda_stream
    if op == "lookup":
        plan.embed_lookup(1, s["buffer"].data_ptr(), s["ids"].data_ptr(), case["tokens"], s["out"].data_ptr(),
                          id_type=s["id_type"], out_type=s["out_type"], first_id=case["first"], scale=case["scale"],
                          stream=stream)
        return s["out"]
    if op == "embed":
        plan.embed_grad(1, s["buffer"].data_ptr(), s["ids"].data_ptr(), case["tokens"], s["dout"].data_ptr(),
                        s["space"].data_ptr(), s["space"].numel(), id_type=s["id_type"], dout_type=s["out_type"],
                        first_id=case["first"], scale=case["scale"], accumulate=case["add"], stream=stream)
        return s["weight"]
    grads, space, flags = s["grads"].data_ptr(), s["space"].data_ptr(), s["flags"]
    stats = s["stats"]
    plan.grad_norm(grads, space, s["space"].numel(), stats.data_ptr(), max_norm=case["max_norm"], eps=EPS,
                   entry_norms=s["norms"].data_ptr() if op == "norm" else 0, stream=stream, flags=flags)
    factor = stats.data_ptr() + 12
    if op == "clip":
        plan.grad_clip(grads, s["out"].data_ptr(), factor, space, s["space"].numel(), stream=stream,
                       flags=s["resident"])
    if op == "step":
        plan.step_scaled(s["params"].data_ptr(), grads, s["state"].data_ptr(), s["step_space"].data_ptr(),
                         s["step_space"].numel(), s["step"], factor, stream=stream, flags=flags)
    s["flags"] = s["resident"]  # the workspaces hold the plan's descriptors from the first pass on
    if op == "norm":
        return [s["norms"], stats[2:4]]
    if op == "clip":
        return [stats[2:4]] + [s["out"][lo:hi].view(dt) for dt, lo, hi, *_ in s["groups"]]
    return [stats[2:4], s["params"].view(s["groups"][0][0]), s["state"]]


def run(state):
    return _own(state) if own else _plain(state)


# ---- what one pass cannot do without ----

def _touched(case):
    """Rows of the table that a batch is expected to touch."""
    rank = np.arange(1, case["rows"] + 1, dtype=np.float64)
    p = (np.log(rank + 1) - np.log(rank)) / math.log(case["rows"] + 1)
    return float((-np.expm1(case["tokens"] * (1 - case["outside"]) * np.log1p(-np.minimum(p, 1 - 1e-12)))).sum())


def work(case):
    op = case["op"]
    if op in ("lookup", "embed"):
        n, d = case["tokens"], case["cols"]
        es, eo = DTYPES[case["table"]].itemsize, DTYPES[case["out"]].itemsize
        rows, inside = _touched(case), n * (1 - case["outside"])
        ids = n * DTYPES[case["ids"]].itemsize
        if op == "lookup":
            return {"bytes": ids + rows * d * es + n * d * eo, "flops": inside * d}
        written = 2 * rows if case["add"] else case["rows"]
        return {"bytes": ids + inside * d * eo + written * d * es, "flops": (inside + rows) * d}
    tensors = _tensors(case["table"])
    size = sum(r * c * DTYPES[d].itemsize for d, r, c in tensors)
    numel = sum(r * c for _, r, c in tensors)
    if op == "norm":
        return {"bytes": size + 4 * len(tensors) + 16, "flops": 2 * numel}
    if op == "clip":
        return {"bytes": 2 * size + 16, "flops": 3 * numel}
    return {"bytes": 3 * size + 16 * numel + 16, "flops": 18 * numel}


# ---- the definition in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("lookup", "embed"):
        rows, d = case["rows"], case["cols"]
        ids = s["ids"].cpu().numpy().astype(np.int64) - case["first"]
        held = np.nonzero((ids >= 0) & (ids < rows))[0]
        where = torch.from_numpy(held).cuda()
        if case["op"] == "lookup":
            out = torch.zeros(case["tokens"], d, dtype=torch.float64, device="cuda")
            out[where] = s["weight"].double()[torch.from_numpy(ids[held]).cuda()] * case["scale"]
            return out
        # positions in the order of their ids; the sum over an id's run is a difference of running sums
        order = held[np.argsort(ids[held], kind="stable")]
        sums = s["weight"].double() if case["add"] else torch.zeros(rows, d, dtype=torch.float64, device="cuda")
        if len(order):
            key = ids[order]
            last = np.nonzero(np.append(key[1:] != key[:-1], True))[0]
            upto = s["dout"][torch.from_numpy(order).cuda()].double().cumsum(0)[torch.from_numpy(last).cuda()]
            upto[1:] -= upto[:-1].clone()
            sums[torch.from_numpy(key[last]).cuda()] += upto * case["scale"]
        return sums
    tensors, (offs, _) = s["tensors"], _layout(s["tensors"])
    take = lambda buf, i: buf[offs[i]:offs[i] + tensors[i][1] * tensors[i][2] * DTYPES[tensors[i][0]].itemsize].view(DTYPES[tensors[i][0]])  # noqa: E731
    sq = [float(torch.linalg.vector_norm(take(s["grads"], i).double())) ** 2 for i in range(len(tensors))]
    norm = math.sqrt(math.fsum(sq))
    factor = min(1.0, case["max_norm"] / (norm + EPS))
    stats = np.array([norm, factor])
    if case["op"] == "norm":
        return [np.sqrt(np.array(sq)), stats]
    if case["op"] == "clip":
        outs = []
        for dt, lo, hi, mask, last, first, rows in s["groups"]:
            o = torch.zeros((hi - lo) // dt.itemsize, dtype=torch.float64, device="cuda")
            for i in range(first, first + len(rows)):
                g = take(s["grads"], i)
                at = (offs[i] - lo) // dt.itemsize
                o[at:at + len(g)] = g.double() * factor
            outs.append(o)
        return [stats] + outs
    w, state = s["params"].view(s["groups"][0][0]).double(), s["state"].double()
    es, at = DTYPES[tensors[0][0]].itemsize, 0
    for i in range(len(tensors)):
        n = tensors[i][1] * tensors[i][2]
        cell = -(-n * 4 // ALIGN) * 64
        g = take(s["grads"], i).double() * factor
        m, v = state[at:at + n], state[at + cell:at + cell + n]
        m.mul_(ADAM["beta1"]).add_(g, alpha=1 - ADAM["beta1"])
        v.mul_(ADAM["beta2"]).addcmul_(g, g, value=1 - ADAM["beta2"])
        p = w[offs[i] // es:offs[i] // es + n]
        move = (m / (1 - ADAM["beta1"] ** s["step"])) / ((v / (1 - ADAM["beta2"] ** s["step"])).sqrt() + ADAM["eps"])
        p.mul_(1 - ADAM["lr"] * ADAM["weight_decay"]).sub_(move, alpha=ADAM["lr"])
        at += 2 * cell
    return [stats, w, state]
