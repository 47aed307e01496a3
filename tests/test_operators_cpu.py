"""Host-side checks of the gradient and embedding operators: struct layouts,
workspace sizes, and every refusal.  Each refused call returns before any HIP
call, so no GPU is needed (the addresses are never read)."""

import ctypes
import math
import os
import shutil
import subprocess
import threading

import pytest

from matrix_optimizer_owner_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E = B.TableEntry
ADDR = 1 << 20  # an aligned address that no refused call may touch
INVALID, UNSUPPORTED, TOO_SMALL = 1, 4, 5


def _plan(entries=None, pbytes=1 << 24):
    entries = [E(0, 40, 50), E(1 << 16, 1, 77, B.F32), E(1 << 17, 0, 5), E(1 << 18, 100, 12, B.F32, B.ROLE_ADAMW)] \
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
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "abi_sizes_operators.c"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split("\n")
    mirrors = {"mfsdp_grad_stats": B.GradStats, "mfsdp_grad_norm_args": B.GradNormArgs,
               "mfsdp_grad_clip_args": B.GradClipArgs, "mfsdp_embed_lookup_args": B.EmbedLookupArgs,
               "mfsdp_embed_grad_args": B.EmbedGradArgs}
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
    assert B.GradStats.scale.offset == B.GradStats.SCALE_OFFSET


def test_grad_workspace_sizes():
    assert _plan([]).grad_workspace_bytes > 0
    small, large = _plan().grad_workspace_bytes, _plan([E(0, 4096, 4096)], 1 << 25).grad_workspace_bytes
    assert 0 < small <= large < 1 << 20
    # the work list stays short for a large table: 872 M elements
    p = _plan([E(i << 27, 4096, 14336) for i in range(15)], 1 << 31)
    assert p.grad_workspace_bytes < 1 << 20


def test_grad_tables_from_two_threads():
    """The plan's work list is built once, whoever asks first."""
    p = _plan()
    got = []
    ts = [threading.Thread(target=lambda: got.append(p.grad_workspace_bytes)) for _ in range(8)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert len(got) == 8 and len(set(got)) == 1


def test_grad_tables_cover_every_element_once(tmp_path):
    """The work lists of 309 tables (empty, single elements, 40000 tensors, 4 TiB, random ones) in C++."""
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("g++ not available")
    csrc = os.path.join(ROOT, "matrix_optimizer_owner_amd", "csrc")
    exe = str(tmp_path / "check")
    subprocess.run([gxx, "-std=c++17", "-O1", "-pthread", "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(csrc, "plan.cpp"), os.path.join(csrc, "grad_plan.cpp"),
                    os.path.join(ROOT, "tests", "grad_plan_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.startswith("OK 309"), out.stdout


def test_clip_work_list_launches_few_empty_blocks(tmp_path):
    """Blocks of a clip against the slices that hold elements, for 118 tables of up to 100000 tensors, in C++."""
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("g++ not available")
    csrc = os.path.join(ROOT, "matrix_optimizer_owner_amd", "csrc")
    exe = str(tmp_path / "check")
    subprocess.run([gxx, "-std=c++17", "-O1", "-pthread", "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(csrc, "plan.cpp"), os.path.join(csrc, "grad_plan.cpp"),
                    os.path.join(ROOT, "tests", "clip_plan_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.startswith("OK 118"), out.stdout


def test_grad_norm_refusals():
    p = _plan()
    ws = p.grad_workspace_bytes
    ok = dict(grads=ADDR, workspace=ADDR, workspace_bytes=ws, stats=ADDR)
    for bad in (dict(grads=0), dict(grads=ADDR + 8), dict(workspace=0), dict(workspace=ADDR + 128), dict(stats=0),
                dict(stats=ADDR + 8), dict(entry_norms=ADDR + 2), dict(max_norm=0.0), dict(max_norm=-1.0),
                dict(max_norm=math.nan), dict(eps=-1e-6), dict(eps=math.inf), dict(eps=math.nan), dict(flags=2)):
        assert _status(p.grad_norm, **dict(ok, **bad)) == INVALID, bad
    assert _status(p.grad_norm, **dict(ok, workspace_bytes=ws - 1)) == TOO_SMALL
    lib = B.load()
    assert lib.mfsdp_grad_norm(None, ctypes.byref(B.GradNormArgs())) == INVALID
    assert lib.mfsdp_grad_norm(p._h, None) == INVALID
    assert lib.mfsdp_plan_grad_workspace_bytes(p._h, None) == INVALID
    assert lib.mfsdp_plan_grad_workspace_bytes(None, ctypes.byref(ctypes.c_uint64())) == INVALID


def test_grad_total_refusals():
    for bad in (dict(parts=0), dict(parts=ADDR + 8), dict(stats=0), dict(stats=ADDR + 4), dict(count=0),
                dict(count=-1), dict(count=65537), dict(max_norm=0.0), dict(eps=-1.0)):
        assert _status(B.grad_total, **dict(dict(parts=ADDR, count=2, stats=ADDR), **bad)) == INVALID, bad


def test_grad_clip_refusals():
    p = _plan()
    ws = p.grad_workspace_bytes
    ok = dict(grads=ADDR, out=ADDR, scale=ADDR, workspace=ADDR, workspace_bytes=ws)
    end = (1 << 18) + 100 * 12 * 4  # the end of the table's last entry
    for bad in (dict(grads=0), dict(grads=ADDR + 4), dict(out=0), dict(out=ADDR + 8), dict(scale=0),
                dict(scale=ADDR + 1), dict(workspace=0), dict(workspace=ADDR + 16), dict(flags=4),
                dict(out=ADDR + 16), dict(out=ADDR + end - 16), dict(out=ADDR - 16)):
        assert _status(p.grad_clip, **dict(ok, **bad)) == INVALID, bad
    assert _status(p.grad_clip, **dict(ok, workspace_bytes=ws - 1)) == TOO_SMALL
    assert B.load().mfsdp_grad_clip(None, ctypes.byref(B.GradClipArgs())) == INVALID
    assert B.load().mfsdp_grad_clip(p._h, None) == INVALID


def test_step_scaled_refusals():
    p = _plan()
    ok = dict(params=ADDR, grads=ADDR, state=ADDR, workspace=ADDR, workspace_bytes=p.workspace_bytes, step=1,
              grad_scale=ADDR)
    for bad in (dict(grad_scale=0), dict(grad_scale=ADDR + 2), dict(params=0), dict(grads=0), dict(state=0),
                dict(workspace=0), dict(step=0), dict(workspace=ADDR + 8)):
        assert _status(p.step_scaled, **dict(ok, **bad)) == INVALID, bad
    assert _status(p.step_scaled, **dict(ok, workspace_bytes=16)) == TOO_SMALL
    assert B.load().mfsdp_owner_step_scaled(p._h, None, ADDR) == INVALID
    assert B.load().mfsdp_owner_step_scaled(None, ctypes.byref(B.StepArgs()), ADDR) == INVALID


def test_embed_lookup_refusals():
    p = _plan()
    ok = dict(entry=3, params=ADDR, ids=ADDR, n_ids=4, out=ADDR)
    for bad in (dict(entry=-1), dict(entry=4), dict(params=0), dict(params=ADDR + 8), dict(ids=0), dict(ids=ADDR + 4),
                dict(out=0), dict(out=ADDR + 1), dict(out=ADDR + 2, out_type=B.F32), dict(ids=ADDR + 2, id_type=B.I32),
                dict(n_ids=-1), dict(n_ids=(1 << 30) + 1), dict(first_id=-1), dict(first_id=(1 << 62) + 1),
                dict(out_stride=11), dict(out_stride=-12), dict(out_stride=(1 << 40) + 1)):
        assert _status(p.embed_lookup, **dict(ok, **bad)) == INVALID, bad
    for bad in (dict(id_type=2), dict(id_type=-1), dict(out_type=2), dict(out_type=7)):
        assert _status(p.embed_lookup, **dict(ok, **bad)) == UNSUPPORTED, bad
    assert _status(p.embed_lookup, **dict(ok, n_ids=0, ids=0, out=0)) == 0  # nothing to do
    assert B.load().mfsdp_embed_lookup(p._h, 3, None) == INVALID
    assert B.load().mfsdp_embed_lookup(None, 3, ctypes.byref(B.EmbedLookupArgs())) == INVALID


def test_embed_grad_refusals():
    p = _plan()
    n = 50_000
    ws = p.embed_workspace_bytes(3, n)
    ok = dict(entry=3, grads=ADDR, ids=ADDR, n_ids=n, dout=ADDR, workspace=ADDR, workspace_bytes=ws)
    for bad in (dict(entry=-1), dict(entry=4), dict(grads=0), dict(grads=ADDR + 8), dict(ids=0), dict(ids=ADDR + 4),
                dict(dout=0), dict(dout=ADDR + 1), dict(dout=ADDR + 2, dout_type=B.F32),
                dict(ids=ADDR + 2, id_type=B.I32), dict(n_ids=-1), dict(n_ids=(1 << 30) + 1), dict(first_id=-1),
                dict(first_id=(1 << 62) + 1), dict(dout_stride=11), dict(dout_stride=-1)):
        assert _status(p.embed_grad, **dict(ok, **bad)) == INVALID, bad
    for bad in (dict(id_type=2), dict(dout_type=2)):
        assert _status(p.embed_grad, **dict(ok, **bad)) == UNSUPPORTED, bad
    if ws:
        assert _status(p.embed_grad, **dict(ok, workspace=0)) == INVALID
        assert _status(p.embed_grad, **dict(ok, workspace=ADDR + 64)) == INVALID
        assert _status(p.embed_grad, **dict(ok, workspace_bytes=ws - 1)) == TOO_SMALL
    a = B.EmbedGradArgs(ADDR, ADDR, 4, B.I64, B.BF16, 0, ADDR, 0, 1.0, 2, ADDR, 1 << 20, None)
    assert B.load().mfsdp_embed_grad(p._h, 3, ctypes.byref(a)) == INVALID  # accumulate is 0 or 1
    assert B.load().mfsdp_embed_grad(p._h, 3, None) == INVALID
    assert B.load().mfsdp_embed_grad(None, 3, ctypes.byref(a)) == INVALID
    # nothing to do: an empty entry, or no ids added to what is there
    assert _status(p.embed_grad, **dict(ok, entry=2)) == 0
    assert _status(p.embed_grad, **dict(ok, n_ids=0, ids=0, dout=0, accumulate=True, workspace=0, workspace_bytes=0)) == 0


def test_none_is_a_null_address():
    """None stands for NULL in the operators' calls as it does in the step's: a refusal or a call that needs none."""
    p = _plan()
    ws = p.grad_workspace_bytes
    norm = dict(grads=ADDR, workspace=ADDR, workspace_bytes=ws, stats=ADDR)
    clip = dict(grads=ADDR, out=ADDR, scale=ADDR, workspace=ADDR, workspace_bytes=ws)
    step = dict(params=ADDR, grads=ADDR, state=ADDR, workspace=ADDR, workspace_bytes=p.workspace_bytes, step=1,
                grad_scale=ADDR)
    lookup = dict(entry=3, params=ADDR, ids=ADDR, n_ids=4, out=ADDR)
    embed = dict(entry=3, grads=ADDR, ids=ADDR, n_ids=50_000, dout=ADDR, workspace=ADDR, workspace_bytes=1 << 30)
    for fn, ok, names in ((p.grad_norm, norm, ("grads", "workspace", "stats")),
                          (p.grad_clip, clip, ("grads", "out", "scale", "workspace")),
                          (p.step_scaled, step, ("params", "grads", "state", "workspace", "grad_scale")),
                          (p.embed_lookup, lookup, ("params", "ids", "out")),
                          (p.embed_grad, embed, ("grads", "ids", "dout", "workspace"))):
        for name in names:
            assert _status(fn, **dict(ok, **{name: None, "stream": None})) == INVALID, (fn, name)
    assert _status(p.grad_norm, **dict(norm, entry_norms=None, stream=None, max_norm=0.0)) == INVALID
    empty = _plan([E(0, 0, 5)])  # nothing to step: the call returns before any HIP call
    assert _status(empty.step_scaled, **dict(step, stream=None, ns_out=None)) == 0
    assert _status(empty.step, **{k: v for k, v in step.items() if k != "grad_scale"}, stream=None, ns_out=None) == 0
    assert _status(p.embed_lookup, **dict(lookup, n_ids=0, ids=None, out=None, stream=None)) == 0
    assert _status(p.embed_grad, **dict(embed, n_ids=0, ids=None, dout=None, accumulate=True, workspace=None,
                                        workspace_bytes=0, stream=None)) == 0


def test_embed_workspace_sizes():
    p = _plan()
    assert p.embed_workspace_bytes(3, 0) == 0
    for bad in ((-1, 5), (4, 5), (3, -1), (3, (1 << 30) + 1)):
        assert _status(p.embed_workspace_bytes, *bad) == INVALID


@pytest.mark.parametrize("rows,cols", [(100, 12), (5000, 64), (300000, 515), (1 << 22, 3), (1000, 4096), (257, 20000),
                                       (128256, 4096)])
def test_embed_workspace_for_more_ids_serves_fewer(rows, cols):
    """What a batch needs never falls as the batch grows."""
    p = _plan([E(0, rows, cols, B.BF16, B.ROLE_ADAMW)], rows * cols * 2)
    sizes = sorted({int(1.07 ** k) + d for k in range(300) for d in (-1, 0, 1)} |
                   {2 ** k + d for k in range(30) for d in (-1, 0, 1)})
    last = 0
    for n in [s for s in sizes if 0 <= s <= 1 << 30]:
        b = p.embed_workspace_bytes(0, n)
        assert b >= last, n
        last = b
