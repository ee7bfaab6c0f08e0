"""CPU tests of include/gated_delta.h: declared functions are exported, structures
have the header's fields, bad arguments are refused on the host before any
launch, sizes add up, and the binding refuses tensors that do not fit."""
import ctypes
import os
import re

import pytest
import torch

import chunked_linear_scan_amd as cls

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gated_delta.h")

pytestmark = pytest.mark.skipif(not os.path.exists(cls.LIB_PATH),
                                reason="library not built (run __graft_entry__.build())")

AT = 0x10000  # 16-byte aligned, never dereferenced on error paths
I64, I32, VP, SZ, F32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, UNSUPPORTED = -1, -2, -3, -5, -6, -8


def struct(name, *groups):
    return type(name, (ctypes.Structure,), {"_fields_": [(n, t) for t, names in groups for n in names.split()]})


DeltaInputs = struct("gated_delta_inputs", (I64, "batch seqlen kheads heads dk dv"), (I32, "dtype"), (F32, "scale"),
                     (VP, "q k v g beta h0 seqlens"),
                     (I64, "q_batch q_token q_head k_batch k_token k_head v_batch v_token v_head g_batch g_token "
                           "beta_batch beta_token"))
DeltaGrads = struct("gated_delta_grads", (VP, "dy"), (I64, "dy_batch dy_token dy_head"),
                    (VP, "dh_final checkpoints dq dk dv dg dbeta dh0"))
NormInputs = struct("gated_norm_inputs", (I64, "rows heads dim"), (I32, "dtype gate_first"), (F32, "eps"),
                    (VP, "x z weight"), (I64, "x_row x_head z_row z_head"))
ResInputs = struct("residual_norm_inputs", (I64, "rows dim"), (I32, "dtype stream_dtype"), (F32, "eps"),
                   (VP, "x residual scale weight"), (I64, "x_row residual_row"))
ResGrads = struct("residual_norm_grads", (VP, "dy dr r rstd"), (I64, "dy_row dr_row r_row"),
                  (VP, "dresidual dx dweight dscale"))


def library():
    lib = ctypes.CDLL(cls.LIB_PATH)
    for name, args, res in (
            ("gated_delta_chunk", [ctypes.c_int], I64), ("gated_delta_workspace_size", [VP], SZ),
            ("gated_delta_bwd_workspace_size", [VP], SZ), ("gated_delta_checkpoint_size", [VP], SZ),
            ("gated_delta_fwd", [VP] * 5 + [SZ, VP], ctypes.c_int), ("gated_delta_bwd", [VP] * 3 + [SZ, VP], ctypes.c_int),
            ("gated_delta_step", [VP] * 4, ctypes.c_int), ("gated_norm_fwd", [VP] * 4, ctypes.c_int),
            ("gated_norm_bwd_workspace_size", [I64] * 3, SZ),
            ("gated_norm_bwd", [VP, VP, I64, I64] + [VP] * 5 + [SZ, VP], ctypes.c_int),
            ("residual_norm_fwd", [VP] * 5, ctypes.c_int), ("residual_norm_bwd_workspace_size", [I64] * 2, SZ),
            ("residual_norm_bwd", [VP] * 3 + [SZ, VP], ctypes.c_int)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res
    return lib


def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_library_exports_every_declared_symbol():
    names = set(re.findall(r"\b([a-z_][a-z0-9_]*)\s*\(", header()))
    assert names == {"gated_delta_chunk", "gated_delta_workspace_size", "gated_delta_bwd_workspace_size",
                     "gated_delta_checkpoint_size", "gated_delta_fwd", "gated_delta_bwd", "gated_delta_step",
                     "gated_norm_fwd", "gated_norm_bwd_workspace_size", "gated_norm_bwd", "residual_norm_fwd",
                     "residual_norm_bwd_workspace_size", "residual_norm_bwd"}
    lib = ctypes.CDLL(cls.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("s", [DeltaInputs, DeltaGrads, NormInputs, ResInputs, ResGrads])
def test_structures_have_the_header_s_fields(s):
    body = re.search(r"typedef struct \{([^}]*)\} %s;" % s.__name__, header()).group(1)
    fields = [re.sub(r"\W", "", f.split()[-1]) for d in body.split(";") for f in d.split(",") if f.strip()]
    assert fields == [f for f, _ in s._fields_]


def delta_in(**k):
    a = dict(batch=2, seqlen=200, kheads=2, heads=4, dk=64, dv=48, dtype=1, scale=1.0, q=AT, k=AT, v=AT, g=AT, beta=AT,
             h0=AT, seqlens=AT, q_batch=200 * 128, q_token=128, q_head=64, k_batch=200 * 128, k_token=128, k_head=64,
             v_batch=200 * 192, v_token=192, v_head=48, g_batch=800, g_token=4, beta_batch=800, beta_token=4)
    a.update(k)
    return DeltaInputs(**a)


BAD = [(dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(g=None), NULL), (dict(beta=None), NULL),
       (dict(dtype=3), DTYPE), (dict(dtype=-1), DTYPE), (dict(batch=0), SHAPE), (dict(kheads=0), SHAPE),
       (dict(heads=0), SHAPE), (dict(heads=3), SHAPE), (dict(dk=0), SHAPE), (dict(dv=0), SHAPE),
       (dict(dk=257), UNSUPPORTED), (dict(dv=65537), UNSUPPORTED), (dict(q=AT + 1), ALIGN), (dict(v=AT + 1), ALIGN),
       (dict(g=AT + 2), ALIGN), (dict(beta=AT + 1), ALIGN), (dict(q_head=-1), SHAPE), (dict(v_batch=-4), SHAPE),
       (dict(g_batch=-1), SHAPE), (dict(k_head=(1 << 40) + 1), SHAPE), (dict(batch=(1 << 20) + 1), SHAPE),
       (dict(heads=1 << 21), SHAPE), (dict(batch=1 << 20, heads=1 << 4), SHAPE)]
BAD_LENGTH = [(dict(seqlen=0), SHAPE), (dict(seqlen=(1 << 30) + 1), SHAPE), (dict(seqlens=AT + 2), ALIGN),
              (dict(h0=AT + 2), ALIGN), (dict(q_token=-1), SHAPE), (dict(g_token=-1), SHAPE),
              (dict(seqlen=1 << 30), SHAPE)]
GRADS = {k: AT for k in ("dy", "checkpoints", "dq", "dk", "dv", "dg", "dbeta")}


@pytest.mark.parametrize("bad,status", BAD + BAD_LENGTH)
def test_delta_refuses(bad, status):
    lib, ref = library(), ctypes.byref(delta_in(**bad))
    assert lib.gated_delta_fwd(ref, AT, AT, AT, AT, 1 << 60, None) == status
    assert lib.gated_delta_bwd(ref, ctypes.byref(DeltaGrads(**GRADS)), AT, 1 << 60, None) == status


@pytest.mark.parametrize("bad,status", BAD)
def test_step_refuses(bad, status):
    assert library().gated_delta_step(ctypes.byref(delta_in(**bad)), AT, AT, None) == status


def test_delta_refuses_other_pointers():
    lib, s = library(), delta_in()
    ref, big = ctypes.byref(s), 1 << 60
    assert lib.gated_delta_fwd(None, AT, AT, AT, AT, big, None) == NULL
    assert lib.gated_delta_fwd(ref, None, AT, AT, AT, big, None) == NULL
    assert lib.gated_delta_fwd(ref, AT + 1, AT, AT, AT, big, None) == ALIGN
    assert lib.gated_delta_fwd(ref, AT, AT + 2, AT, AT, big, None) == ALIGN
    assert lib.gated_delta_fwd(ref, AT, AT, AT + 8, AT, big, None) == ALIGN
    assert lib.gated_delta_fwd(ref, AT, AT, AT, AT + 8, big, None) == ALIGN
    need = lib.gated_delta_workspace_size(ref)
    assert need > 0
    assert lib.gated_delta_fwd(ref, AT, AT, AT, AT, need - 1, None) == WORKSPACE
    assert lib.gated_delta_fwd(ref, AT, AT, AT, None, big, None) == WORKSPACE
    for k in GRADS:
        g = DeltaGrads(**{**GRADS, k: None})
        assert lib.gated_delta_bwd(ref, ctypes.byref(g), AT, big, None) == NULL, k
    for k, v, st in (("dq", AT + 1, ALIGN), ("dy", AT + 1, ALIGN), ("dg", AT + 2, ALIGN), ("dh0", AT + 2, ALIGN),
                     ("dh_final", AT + 1, ALIGN), ("checkpoints", AT + 4, ALIGN), ("dy_token", -2, SHAPE)):
        g = DeltaGrads(**{**GRADS, k: v})
        assert lib.gated_delta_bwd(ref, ctypes.byref(g), AT, big, None) == st, k
    g = ctypes.byref(DeltaGrads(**GRADS))
    need = lib.gated_delta_bwd_workspace_size(ref)
    assert lib.gated_delta_bwd(ref, g, AT, need - 1, None) == WORKSPACE
    assert lib.gated_delta_bwd(ref, g, None, big, None) == WORKSPACE
    assert lib.gated_delta_bwd(ref, None, AT, big, None) == NULL
    assert lib.gated_delta_step(None, AT, AT, None) == NULL
    assert lib.gated_delta_step(ref, None, AT, None) == NULL
    assert lib.gated_delta_step(ref, AT, None, None) == NULL
    assert lib.gated_delta_step(ref, AT + 8, AT, None) == ALIGN  # dk is whole vectors
    assert lib.gated_delta_step(ctypes.byref(delta_in(dk=63)), AT + 2, AT, None) == ALIGN


# a misaligned output is what is refused after the sizes
LIMITS = [(dict(batch=1 << 20, seqlen=1, heads=6), SHAPE), (dict(batch=1 << 20, seqlen=1, kheads=1, heads=3), ALIGN), (dict(batch=1 << 20, seqlen=64, heads=16), SHAPE),
          (dict(batch=1, seqlen=1 << 30, kheads=1, heads=1), SHAPE), (dict(batch=1, seqlen=(1 << 30) - 64, kheads=1, heads=1), ALIGN),
          (dict(batch=1, seqlen=(1 << 29) - 32, kheads=1, heads=1, dtype=0), ALIGN),
          (dict(batch=1, seqlen=1 << 29, kheads=1, heads=1, dtype=0), SHAPE),
          (dict(batch=1 << 12, seqlen=1, kheads=1, heads=1, dv=65536), SHAPE),
          (dict(batch=(1 << 12) - 1, seqlen=1, kheads=1, heads=1, dv=65536), ALIGN),
          (dict(batch=1, heads=128, dv=65536), ALIGN), (dict(batch=1, heads=130, dv=65536), SHAPE),  # 2^23 in a token's row
          (dict(batch=1, kheads=1 << 15, heads=1 << 15), ALIGN), (dict(batch=1, kheads=(1 << 15) + 1, heads=(1 << 15) + 1), SHAPE)]


@pytest.mark.parametrize("size,status", LIMITS)
def test_delta_size_limits(size, status):
    lib, ref = library(), ctypes.byref(delta_in(**size))
    assert lib.gated_delta_fwd(ref, AT + 1, AT, AT, AT, 1 << 62, None) == status
    assert (lib.gated_delta_workspace_size(ref) > 0) == (status == ALIGN)
    assert (lib.gated_delta_bwd_workspace_size(ref) > 0) == (status == ALIGN)
    assert (lib.gated_delta_checkpoint_size(ref) > 0) == (status == ALIGN)


def test_shared_key_heads_limit_the_gradients():
    lib = library()
    g = ctypes.byref(DeltaGrads(**{**GRADS, "dq": AT + 1}))
    for seqlen, status in ((1 << 24, SHAPE), ((1 << 24) - 1, ALIGN)):
        s = delta_in(batch=1, seqlen=seqlen, kheads=1, heads=2, dk=256)
        assert lib.gated_delta_bwd(ctypes.byref(s), g, AT, 1 << 62, None) == status
    s = delta_in(batch=1, seqlen=1 << 24, kheads=2, heads=2, dk=256)
    assert lib.gated_delta_bwd(ctypes.byref(s), g, AT, 1 << 62, None) == ALIGN


def test_delta_sizes_add_up():
    lib = library()
    assert [lib.gated_delta_chunk(d) for d in (0, 1, 2, 3)] == [32, 64, 64, 0]
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    for dtype, C, mat in ((1, 64, 4 * 64 * 64 * 2), (0, 32, 2 * 32 * 32 * 4)):
        s = delta_in(dtype=dtype)
        chunks = 2 * 4 * -(-200 // C)
        fwd = up(chunks * mat) + up(chunks * 5 * C * 4)
        states, tokens = up(chunks * 64 * 48 * 4), up(chunks * C * 48 * 4)
        size = 4 if dtype == 0 else 2
        keys, values = up(2 * 200 * 2 * 64 * size), up(2 * 200 * 4 * 48 * size)
        assert lib.gated_delta_workspace_size(ctypes.byref(s)) == fwd
        assert lib.gated_delta_checkpoint_size(ctypes.byref(s)) == states + tokens
        assert lib.gated_delta_bwd_workspace_size(ctypes.byref(s)) == fwd + states + tokens + 2 * up(2 * 200 * 4 * 64 * 4) + values
        # rows that the kernels cannot read in place are copied: those off whole vectors (q and k), and of other strides
        for bad, more in ((dict(q=AT + 8), keys), (dict(k_head=63), keys), (dict(v=AT + 4), values), (dict(v_token=47), values),
                          (dict(v_token=(1 << 23) + 8), values), (dict(q_token=0, k_token=8), 2 * keys),
                          (dict(seqlen=1, q_token=0, k_token=0, v_token=0), None)):
            s = delta_in(dtype=dtype, **bad)
            if more is None:
                assert lib.gated_delta_workspace_size(ctypes.byref(s)) == up(8 * mat) + up(8 * 5 * C * 4)
            else:
                assert lib.gated_delta_workspace_size(ctypes.byref(s)) == fwd + more, bad
        s = delta_in(dtype=dtype, kheads=4)
        assert lib.gated_delta_bwd_workspace_size(ctypes.byref(s)) == fwd + states + tokens + values


def norm_in(**k):
    return NormInputs(**{**dict(rows=7, heads=3, dim=64, dtype=1, eps=1e-6, x=AT, z=AT, weight=AT, x_row=192, x_head=64,
                                z_row=192, z_head=64), **k})


@pytest.mark.parametrize("bad,status", [(dict(x=None), NULL), (dict(dtype=4), DTYPE), (dict(rows=0), SHAPE),
                                        (dict(heads=0), SHAPE), (dict(dim=0), SHAPE), (dict(dim=16385), UNSUPPORTED),
                                        (dict(rows=1 << 31), SHAPE), (dict(rows=1 << 30, heads=2), SHAPE),
                                        (dict(x=AT + 1), ALIGN), (dict(z=AT + 1), ALIGN), (dict(weight=AT + 2), ALIGN),
                                        (dict(x_row=-1), SHAPE), (dict(z_head=-1), SHAPE)])
def test_gated_norm_refuses(bad, status):
    lib, ref = library(), ctypes.byref(norm_in(**bad))
    assert lib.gated_norm_fwd(ref, AT, AT, None) == status
    assert lib.gated_norm_bwd(ref, AT, 0, 0, AT, AT, AT, AT, AT, 1 << 60, None) == status


def test_gated_norm_refuses_other_pointers():
    lib, ref, big = library(), ctypes.byref(norm_in()), 1 << 60
    assert lib.gated_norm_fwd(None, AT, AT, None) == NULL
    assert lib.gated_norm_fwd(ref, None, AT, None) == NULL
    assert lib.gated_norm_fwd(ref, AT + 1, AT, None) == ALIGN
    assert lib.gated_norm_fwd(ref, AT, AT + 2, None) == ALIGN
    ok = [AT, 0, 0, AT, AT, AT, AT, AT, big, None]
    for at, v, st in ((0, None, NULL), (3, None, NULL), (4, None, NULL), (5, None, NULL), (7, None, WORKSPACE), (1, -1, SHAPE),
                      (4, AT + 1, ALIGN), (6, AT + 2, ALIGN), (7, AT + 4, ALIGN),
                      (8, lib.gated_norm_bwd_workspace_size(7, 3, 64) - 1, WORKSPACE)):
        args = list(ok)
        args[at] = v
        assert lib.gated_norm_bwd(ref, *args) == st, at
    assert lib.gated_norm_bwd_workspace_size(7, 3, 64) == 64 * 4  # one workgroup walks 32 rows of 64
    assert lib.gated_norm_bwd_workspace_size(100000, 1, 5120) == 256 * 5120 * 4  # a workgroup has 1024 lanes
    assert lib.gated_norm_bwd_workspace_size(1, 1, 16385) == 0


def res_in(**k):
    return ResInputs(**{**dict(rows=7, dim=64, dtype=1, stream_dtype=0, eps=1e-6, x=AT, residual=AT, scale=AT, weight=AT,
                               x_row=64, residual_row=64), **k})


RES = {k: AT for k in ("dy", "r", "rstd", "dresidual", "dx", "dweight", "dscale")}


@pytest.mark.parametrize("bad,status", [(dict(dtype=4), DTYPE), (dict(stream_dtype=2), DTYPE), (dict(rows=0), SHAPE),
                                        (dict(dim=0), SHAPE), (dict(dim=16385), UNSUPPORTED), (dict(rows=1 << 31), SHAPE),
                                        (dict(x=AT + 1), ALIGN), (dict(residual=AT + 2), ALIGN), (dict(scale=AT + 2), ALIGN),
                                        (dict(weight=AT + 1), ALIGN), (dict(x_row=-1), SHAPE)])
def test_residual_norm_refuses(bad, status):
    lib, ref = library(), ctypes.byref(res_in(**bad))
    assert lib.residual_norm_fwd(ref, AT, AT, AT, None) == status
    assert lib.residual_norm_bwd(ref, ctypes.byref(ResGrads(**RES)), AT, 1 << 60, None) == status


def test_residual_norm_refuses_other_pointers():
    lib, ref, big = library(), ctypes.byref(res_in()), 1 << 60
    assert lib.residual_norm_fwd(ctypes.byref(res_in(x=None)), AT, AT, AT, None) == NULL
    assert lib.residual_norm_fwd(ref, None, AT, AT, None) == NULL
    assert lib.residual_norm_fwd(ref, AT, None, AT, None) == NULL
    assert lib.residual_norm_fwd(ref, AT + 1, AT, AT, None) == ALIGN
    assert lib.residual_norm_fwd(ref, AT, AT + 2, AT, None) == ALIGN  # the stream is fp32
    for k, v, st in (("dy", None, NULL), ("r", None, NULL), ("rstd", None, NULL), ("dresidual", None, NULL),
                     ("dr_row", -1, SHAPE), ("r", AT + 2, ALIGN), ("dx", AT + 1, ALIGN), ("dscale", AT + 2, ALIGN)):
        g = ResGrads(**{**RES, k: v})
        assert lib.residual_norm_bwd(ref, ctypes.byref(g), AT, big, None) == st, k
    g = ctypes.byref(ResGrads(**RES))
    assert lib.residual_norm_bwd(ctypes.byref(res_in(x=None)), g, AT, big, None) == NULL  # dscale needs x
    need = lib.residual_norm_bwd_workspace_size(7, 64)
    assert need == 2 * 64 * 4
    assert lib.residual_norm_bwd(ref, g, AT, need - 1, None) == WORKSPACE
    assert lib.residual_norm_bwd(ref, g, None, big, None) == WORKSPACE
    assert lib.residual_norm_bwd(None, g, AT, big, None) == NULL
    assert lib.residual_norm_bwd_workspace_size(0, 64) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    q, v, g = torch.zeros(2, 5, 1, 8), torch.zeros(2, 5, 2, 8), torch.zeros(2, 5, 2)
    with pytest.raises(ValueError, match="GPU"):
        cls.gated_delta(q, q, v, g, g)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        cls.gated_delta(q, q, v.double(), g, g)
    with pytest.raises(ValueError, match="batch, seqlen, heads, dv"):
        cls.gated_delta(q, q, v[0], g, g)
    with pytest.raises(ValueError, match="batch, heads, dv"):
        cls.gated_delta_step(v, q, q, v, g, g)
    with pytest.raises(ValueError, match="GPU"):
        cls.gated_norm(v)
    with pytest.raises(ValueError, match="heads, dim"):
        cls.gated_norm(torch.zeros(4))
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        cls.residual_norm(v.int())
    with pytest.raises(ValueError, match="dim"):
        cls.residual_norm(torch.zeros(()))
