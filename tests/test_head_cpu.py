"""Host-side checks of the output head: struct layouts, workspace sizes, and
every refusal.  Each refused call returns before any HIP call, so no GPU is
needed (the addresses are never read)."""

import ctypes
import math
import os
import random
import shutil
import subprocess

import pytest

from matrix_optimizer_owner_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E = B.TableEntry
ADDR = 1 << 20
INVALID, UNSUPPORTED, TOO_SMALL = 1, 4, 5


def _plan(entries=None, pbytes=1 << 24):
    entries = [E(0, 40, 50), E(1 << 16, 1, 77, B.F32), E(1 << 17, 0, 5), E(1 << 18, 100, 12, B.F32, B.ROLE_ADAMW8)] \
        if entries is None else entries
    return B.OwnerPlan(entries, pbytes, B.make_hparams())


def _status(fn, *a, **kw):
    try:
        fn(*a, **kw)
        return 0
    except B.MfsdpError as e:
        assert e.message  # every refusal says why
        return e.status


def test_struct_layouts_match_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    exe = str(tmp_path / "abi")
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "abi_sizes_head.c"),
                    "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split("\n")
    mirrors = {"mfsdp_moments_args": B.MomentsArgs, "mfsdp_head_record": B.HeadRecord,
               "mfsdp_head_logprob_args": B.HeadLogprobArgs, "mfsdp_head_total_args": B.HeadTotalArgs,
               "mfsdp_head_grad_args": B.HeadGradArgs}
    seen = {k: set() for k in mirrors}
    for line in filter(None, out):
        key, val = line.split()
        kind, name = key.split(":")
        if kind == "sizeof":
            assert ctypes.sizeof(mirrors[name]) == int(val), line
        else:
            struct, field = name.split(".")
            assert getattr(mirrors[struct], field).offset == int(val), line
            seen[struct].add(field)
    for name, m in mirrors.items():
        assert seen[name] == {f[0] for f in m._fields_}, name
    assert B.HEAD_RECORD_BYTES == 24


SIZES = [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1000, 2048, 2049, 4096, 5000, 65536, 70000,
         131072, 131073, 1 << 20]


@pytest.mark.parametrize("rows,cols,kind", [(128256, 4096, B.BF16), (50257, 768, B.BF16), (12501, 1001, B.F32), (5, 7, B.F32),
                                            (300, 64, B.BF16), (1, 1, B.BF16), (40000, 130, B.BF16)])
def test_workspace_never_falls_as_the_batch_grows(rows, cols, kind):
    p = _plan([E(0, rows, cols, kind, B.ROLE_ADAMW)], 1 << 34)
    rng = random.Random(rows)
    sizes = sorted(set([n for n in SIZES if n * rows < 2 ** 37] + [rng.randint(1, 9000) for _ in range(200)]))
    for x_type in (B.F32, B.BF16):
        for top_k, grad in ((0, False), (5, False), (0, True), (64, True)):
            need = [p.head_workspace_bytes(0, n, x_type=x_type, top_k=top_k, grad=grad) for n in sizes]
            assert all(a <= b for a, b in zip(need, need[1:]))
            assert need[0] > 0
            if grad:  # serves the call forward too
                assert all(g >= p.head_workspace_bytes(0, n, x_type=x_type, top_k=top_k) for n, g in zip(sizes, need))
    assert p.head_workspace_bytes(0, 0) == 0


def test_workspace_sizes_of_an_empty_table():
    p = _plan()
    assert p.head_workspace_bytes(2, 100, top_k=3, grad=True) == 0


def test_workspace_refusals():
    p = _plan()
    f = p.head_workspace_bytes
    for entry in (-1, 4):
        assert _status(f, entry, 5) == INVALID
    for n in (-1, (1 << 22) + 1):
        assert _status(f, 0, n) == INVALID
    for k in (-1, 65):
        assert _status(f, 0, 5, top_k=k) == INVALID
    assert _status(f, 0, 5, x_type=2) == UNSUPPORTED
    v = ctypes.c_uint64()
    lib = B.load()
    assert lib.mfsdp_plan_head_workspace_bytes(p._h, 0, 5, B.BF16, 0, 2, ctypes.byref(v)) == INVALID
    assert lib.mfsdp_plan_head_workspace_bytes(p._h, 0, 5, B.BF16, 0, 0, None) == INVALID
    assert lib.mfsdp_plan_head_workspace_bytes(None, 0, 5, B.BF16, 0, 0, ctypes.byref(v)) == INVALID
    wide = _plan([E(0, 2, (1 << 20) + 1, B.BF16)], 1 << 24)
    assert _status(wide.head_workspace_bytes, 0, 5) == UNSUPPORTED
    tall = _plan([E(0, 1 << 22, 4, B.BF16, B.ROLE_ADAMW)], 1 << 26)
    assert _status(tall.head_workspace_bytes, 0, 1 << 22) == UNSUPPORTED
    assert _status(tall.head_workspace_bytes, 0, 1000) == 0
    low = _plan([E(0, 2, 8192, B.BF16)], 1 << 24)
    assert _status(low.head_workspace_bytes, 0, 1 << 22) == UNSUPPORTED  # too many tiles of x
    assert _status(low.head_workspace_bytes, 0, 1 << 21) == 0


def test_logprob_refusals():
    p = _plan()
    need = p.head_workspace_bytes(3, 9, x_type=B.F32, top_k=2)
    ok = dict(entry=3, params=ADDR, x=ADDR, n=9, records=ADDR, workspace=ADDR, workspace_bytes=need, ids=ADDR, x_type=B.F32,
              logp=ADDR, entropy=ADDR, top_k=2, top_ids=ADDR, top_logp=ADDR, top_logits=ADDR)
    for bad in (dict(entry=-1), dict(entry=4), dict(params=0), dict(params=None), dict(params=ADDR + 8), dict(x=0),
                dict(x=ADDR + 2), dict(n=-1), dict(n=(1 << 22) + 1), dict(records=0), dict(records=ADDR + 4),
                dict(workspace=0), dict(workspace=ADDR + 128), dict(ids=ADDR + 4), dict(ids=ADDR + 2, id_type=B.I32),
                dict(logp=ADDR + 2), dict(entropy=ADDR + 1), dict(top_ids=0), dict(top_ids=ADDR + 4), dict(top_logp=ADDR + 2),
                dict(top_logits=ADDR + 2), dict(top_k=-1), dict(top_k=65), dict(x_stride=11), dict(x_stride=(1 << 40) + 1),
                dict(first_id=-1), dict(first_id=(1 << 62) + 1), dict(scale=math.nan), dict(scale=math.inf)):
        assert _status(p.head_logprob, **dict(ok, **bad)) == INVALID, bad
    for bad in (dict(x_type=2), dict(id_type=2), dict(id_type=-1)):
        assert _status(p.head_logprob, **dict(ok, **bad)) == UNSUPPORTED, bad
    assert _status(p.head_logprob, **dict(ok, workspace_bytes=need - 1)) == TOO_SMALL
    assert _status(p.head_logprob, **dict(ok, n=0, x=0, records=0, workspace=0, workspace_bytes=0)) == 0
    lib = B.load()
    assert lib.mfsdp_head_logprob(p._h, 0, None) == INVALID and lib.mfsdp_head_logprob(None, 0, None) == INVALID


def test_total_refusals():
    ok = dict(parts=ADDR, count=2, n=9, records=ADDR, logp=ADDR, entropy=ADDR, top_k=3, part_top_ids=ADDR,
              part_top_logits=ADDR, top_ids=ADDR, top_logp=ADDR, top_logits=ADDR)
    for bad in (dict(parts=0), dict(parts=ADDR + 4), dict(count=0), dict(count=65537), dict(n=-1), dict(n=(1 << 22) + 1),
                dict(records=0), dict(records=ADDR + 4), dict(logp=ADDR + 2), dict(entropy=ADDR + 2), dict(top_k=-1),
                dict(top_k=65), dict(part_top_ids=0), dict(part_top_ids=ADDR + 4), dict(part_top_logits=0),
                dict(part_top_logits=ADDR + 2), dict(top_ids=0), dict(top_ids=ADDR + 4), dict(top_logp=ADDR + 1),
                dict(top_logits=ADDR + 1)):
        assert _status(B.head_total, **dict(ok, **bad)) == INVALID, bad
    assert _status(B.head_total, **dict(ok, n=0, parts=0, records=0)) == 0
    assert B.load().mfsdp_head_total(None) == INVALID


def test_grad_refusals():
    p = _plan()
    need = p.head_workspace_bytes(3, 9, x_type=B.F32, grad=True)
    ok = dict(entry=3, params=ADDR, grads=ADDR, x=ADDR, n=9, records=ADDR, dlogp=ADDR, workspace=ADDR, workspace_bytes=need,
              dentropy=ADDR, dx=ADDR, ids=ADDR, x_type=B.F32)
    for bad in (dict(entry=-1), dict(entry=4), dict(params=0), dict(params=ADDR + 8), dict(grads=ADDR + 8), dict(x=0),
                dict(x=ADDR + 2), dict(n=-1), dict(n=(1 << 22) + 1), dict(records=0), dict(records=ADDR + 4), dict(dlogp=0),
                dict(dlogp=ADDR + 2), dict(dentropy=ADDR + 2), dict(dx=ADDR + 2), dict(workspace=0),
                dict(workspace=ADDR + 128), dict(ids=ADDR + 4), dict(x_stride=11), dict(dx_stride=11), dict(dx_stride=-1),
                dict(dx_stride=(1 << 40) + 1), dict(first_id=-1), dict(scale=math.nan)):
        assert _status(p.head_grad, **dict(ok, **bad)) == INVALID, bad
    for bad in (dict(x_type=2), dict(id_type=2)):
        assert _status(p.head_grad, **dict(ok, **bad)) == UNSUPPORTED, bad
    assert _status(p.head_grad, **dict(ok, workspace_bytes=need - 1)) == TOO_SMALL
    # nothing to do: an empty batch that is added, an empty batch without a gradient to write
    assert _status(p.head_grad, **dict(ok, n=0, x=0, records=0, dlogp=0, workspace=0, accumulate=True)) == 0
    assert _status(p.head_grad, **dict(ok, n=0, x=0, records=0, dlogp=0, workspace=0, grads=0)) == 0
    lib = B.load()
    assert lib.mfsdp_head_grad(p._h, 0, None) == INVALID and lib.mfsdp_head_grad(None, 0, None) == INVALID
    args = B.HeadGradArgs(ADDR, ADDR, 9, 0, B.F32, B.I64, ADDR, 0, 1.0, 2, ADDR, ADDR, ADDR, ADDR, 0, ADDR, ADDR, need, None)
    assert lib.mfsdp_head_grad(p._h, 3, ctypes.byref(args)) == INVALID  # accumulate
