"""Refusals of the operators of kda_layers.h: on the host, before any CUDA call (no GPU needed)."""
import ctypes
import os
import subprocess

import pytest
import torch

# The refusals are called with made-up device addresses: were a check lost, a kernel would run on
# them where a GPU is reachable, so these run only where none is.
host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="made-up device addresses: run only where no GPU can be reached")
ARG, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = -1, -2, -3, -4, -7


@pytest.fixture(scope="module")
def L():
    from gated_delta_rule_73_b200 import build as B
    B.build()
    from gated_delta_rule_73_b200 import layers
    return layers


def _call(L, name, n, dims, opts=None, null=(), at=(), same=()):
    """Status of a call whose n pointers are all good ones, but for `null`, `at` (index, address), `same` (i, j)."""
    p = [(i + 1) << 28 for i in range(n)]
    for i in null:
        p[i] = None
    for i, a in at:
        p[i] = a
    for i, j in same:
        p[i] = p[j]
    return getattr(L._lib, name)(*p, dims, opts, None)


def _conv(L, **kw):
    d = dict(B=2, T=8, D=16, K=4, silu=1)
    return L.kda_conv_dims(**{**d, **kw})


def _ssm(L, **kw):
    d = dict(B=2, T=8, D=16, N=16, G=1, dt_softplus=1)
    return L.kda_ssm_dims(**{**d, **kw})


def _norm(L, **kw):
    return L.kda_norm_dims(**{**dict(rows=4, D=64, eps=1e-5), **kw})


def _opts(L, ws=None, nbytes=0, **kw):
    o = L._opts(torch.bfloat16)
    o.workspace, o.workspace_bytes = ws, nbytes
    for k, v in kw.items():
        setattr(o, k, v)
    return o


@host_only
def test_short_conv_refusals(L):
    fwd = lambda d, **kw: _call(L, "kda_short_conv_fwd", 6, d, **kw)  # noqa: E731
    for bad, st in (({"K": 1}, UNSUPPORTED), ({"K": 5}, UNSUPPORTED), ({"B": -1}, ARG), ({"T": -1}, ARG), ({"D": -8}, ARG),
                    ({"silu": 2}, ARG), ({"ld_x": -16}, ARG), ({"ld_x": 15}, SHAPE), ({"ld_y": 8}, SHAPE),
                    ({"B": 1 << 20, "T": 1 << 20}, SHAPE), ({"ld_x": 1 << 41}, SHAPE), ({"zero_rest": 3}, ARG)):
        assert fwd(_conv(L, **bad)) == st, bad
    for i in (0, 1, 4):
        assert fwd(_conv(L), null=[i]) == ARG
    for i in range(6):   # rows may start at any element, the others at 16 bytes
        assert fwd(_conv(L), at=[(i, (i + 1 << 28) + (8 if i not in (0, 4) else 1))]) == ALIGN
    assert fwd(_conv(L), same=[(4, 0)]) == ARG and fwd(_conv(L), same=[(5, 3)]) == ARG
    assert fwd(_conv(L), opts=_opts(L, flags=2)) == ARG      # a flag of the delta rule
    assert fwd(_conv(L), opts=_opts(L, dtype=5)) == ARG
    assert fwd(None) == ARG
    assert fwd(_conv(L, B=0)) == 0 and fwd(_conv(L, D=0)) == 0
    assert fwd(_conv(L, cu_seqlens=(1 << 28) + 2)) == ALIGN
    # y a row behind x, inside it; beside it in wider rows (refused for its alignment alone, behind the overlap's check)
    assert fwd(_conv(L), at=[(4, (1 << 28) + 32)]) == ARG
    assert fwd(_conv(L, ld_x=32, ld_y=32), at=[(4, (1 << 28) + 16)]) == ARG
    assert fwd(_conv(L, ld_x=32, ld_y=33), at=[(4, (1 << 28) + 32)]) == ARG
    bwd = lambda d, **kw: _call(L, "kda_short_conv_bwd", 10, d, **kw)  # noqa: E731
    need = L._lib.kda_short_conv_bwd_workspace_bytes(_conv(L), None)
    assert need > 0
    assert bwd(_conv(L)) == WORKSPACE
    assert bwd(_conv(L), opts=_opts(L, 1 << 40, need - 1)) == WORKSPACE
    assert bwd(_conv(L), opts=_opts(L, (1 << 40) + 8, need)) == ALIGN
    assert bwd(_conv(L), opts=_opts(L, 1 << 28, need)) == ARG    # the workspace is an input
    for i in (0, 1, 4, 6, 7):
        assert bwd(_conv(L), null=[i], opts=_opts(L, 1 << 40, need)) == ARG
    step = lambda d, **kw: _call(L, "kda_short_conv_step", 6, d, **kw)  # noqa: E731
    for i in (0, 1, 3, 4, 5):
        assert step(_conv(L), null=[i]) == ARG
    assert step(_conv(L), same=[(5, 0)]) == ARG and step(_conv(L), same=[(5, 3)]) == ARG


@host_only
def test_ssm_refusals(L):
    fwd = lambda d, **kw: _call(L, "kda_ssm_scan_fwd", 11, d, **kw)  # noqa: E731
    for bad, st in (({"N": 4}, UNSUPPORTED), ({"N": 24}, UNSUPPORTED), ({"N": 128}, UNSUPPORTED), ({"G": 0}, ARG),
                    ({"G": 3}, SHAPE), ({"B": -1}, ARG), ({"T": -2}, ARG), ({"dt_softplus": 7}, ARG),
                    ({"ld_u": 8}, SHAPE), ({"ld_B": 8}, SHAPE), ({"ld_C": -1}, ARG), ({"B": 1 << 20, "T": 1 << 20}, SHAPE)):
        assert fwd(_ssm(L, **bad)) == st, bad
    for i in (0, 1, 2, 3, 4, 9):
        assert fwd(_ssm(L), null=[i]) == ARG
    for i in range(11):
        assert fwd(_ssm(L), at=[(i, (i + 1 << 28) + (8 if i not in (0, 1, 3, 4, 6, 9) else 1))]) == ALIGN
    assert fwd(_ssm(L), same=[(10, 8)]) == ARG      # h_T over h0
    long = _ssm(L, T=4096)
    need = L._lib.kda_ssm_scan_fwd_workspace_bytes(long, None)
    assert need > 0 and fwd(long) == WORKSPACE
    assert fwd(long, opts=_opts(L, 1 << 40, need - 4)) == WORKSPACE
    bwd = lambda d, **kw: _call(L, "kda_ssm_scan_bwd", 20, d, **kw)  # noqa: E731
    need = L._lib.kda_ssm_scan_bwd_workspace_bytes(_ssm(L), None)
    assert bwd(_ssm(L)) == WORKSPACE and bwd(_ssm(L), opts=_opts(L, 1 << 40, need - 1)) == WORKSPACE
    ok = _opts(L, 1 << 40, need)
    for i in (0, 1, 2, 3, 4, 9, 11, 12, 13, 14, 15):
        assert bwd(_ssm(L), null=[i], opts=ok) == ARG
    assert bwd(_ssm(L), null=[6], opts=ok) == ARG and bwd(_ssm(L), null=[17], opts=ok) == ARG   # z without dz, dz without z
    assert bwd(_ssm(L), same=[(11, 0)], opts=ok) == ARG and bwd(_ssm(L), same=[(11, 12)], opts=ok) == ARG
    step = lambda d, **kw: _call(L, "kda_ssm_step", 11, d, **kw)  # noqa: E731
    for i in (0, 1, 2, 3, 4, 8, 9, 10):
        assert step(_ssm(L), null=[i]) == ARG
    assert step(_ssm(L), same=[(10, 8)]) == ARG
    assert step(_ssm(L), at=[(9, (9 << 28) + 64)]) == ARG   # h_out inside h, not in place
    assert step(_ssm(L, B=0)) == 0


@host_only
def test_norm_refusals(L):
    fwd = lambda d, **kw: _call(L, "kda_block_norm_fwd", 8, d, **kw)  # noqa: E731
    for bad, st in (({"D": 0}, UNSUPPORTED), ({"D": 16385}, UNSUPPORTED), ({"rows": -1}, ARG), ({"eps": -1.0}, ARG),
                    ({"eps": float("nan")}, ARG), ({"eps": float("inf")}, ARG), ({"ld_gate": 63}, SHAPE)):
        assert fwd(_norm(L, **bad)) == st, bad
    assert fwd(_norm(L), null=[0]) == ARG and fwd(_norm(L), null=[6]) == ARG and fwd(_norm(L), null=[6, 7]) == ARG
    assert fwd(_norm(L), null=[1]) == ARG           # no block, but its gate and res_out
    assert fwd(_norm(L), same=[(7, 0)]) == ARG and fwd(_norm(L), same=[(6, 1)]) == ARG
    assert fwd(_norm(L, ld_res=128), same=[(6, 0)]) == ARG    # in place needs contiguous rows
    assert fwd(_norm(L, rows=0)) == 0
    bwd = lambda d, **kw: _call(L, "kda_block_norm_bwd", 14, d, **kw)  # noqa: E731
    need = L._lib.kda_block_norm_bwd_workspace_bytes(_norm(L), None)
    assert bwd(_norm(L)) == WORKSPACE
    ok = _opts(L, 1 << 40, need)
    assert bwd(_norm(L), null=[6, 7], opts=ok) == ARG
    for i in (0, 1, 2, 8, 9, 10):   # also a block without dblock, a gate without dgate and the other way round
        assert bwd(_norm(L), null=[i], opts=ok) == ARG
    assert bwd(_norm(L), same=[(8, 7)], opts=ok) == ARG and bwd(_norm(L), same=[(9, 6)], opts=ok) == ARG


@host_only
def test_scan_sizes_are_bounded_by_the_shortest_spans(L):
    """The seams' states of a backward in spans of 16 rows may be 2^40 values, no more."""
    rows, D, N = 1 << 27, 2048, 64          # D N rows / 16 = 2^40 - and some for the sequence
    for d, st in ((_ssm(L, B=1, T=rows, D=D, N=N), SHAPE), (_ssm(L, B=1, T=rows - 4096, D=D, N=N), WORKSPACE)):
        assert _call(L, "kda_ssm_scan_bwd", 20, d, at=[(i, (i + 1) << 44) for i in range(20)]) == st
        assert (L._lib.kda_ssm_scan_bwd_workspace_bytes(d, None) == 0) == (st == SHAPE)


@host_only
def test_outputs_over_the_largest_table_of_bounds(L):
    """The table of 2^31 - 1 sequences is 8 GB long, to the call's check of what its outputs overlap as well."""
    n, at = (1 << 31) - 1, 1 << 36
    inside = at + (1 << 32)
    for name, pointers, d, out, ok in (
            ("kda_short_conv_fwd", 6, _conv(L, B=n, T=4, cu_seqlens=at), 4, (2, 3, 5)),
            ("kda_short_conv_bwd", 10, _conv(L, B=n, T=4, cu_seqlens=at), 6, (2, 3, 5, 8, 9)),
            ("kda_ssm_scan_fwd", 11, _ssm(L, B=n, T=4, D=2, N=8, cu_seqlens=at), 9, (5, 6, 7, 8, 10)),
            ("kda_ssm_scan_bwd", 20, _ssm(L, B=n, T=4, D=2, N=8, cu_seqlens=at), 11, (5, 7, 8, 10, 16, 18, 19))):
        assert _call(L, name, pointers, d, null=ok, at=[(out, inside)], opts=_opts(L, 1 << 50, 1 << 62)) == ARG, name


def test_binding_refuses_what_the_library_could_not_see(L):
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        L.short_conv_fwd(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        L.ssm_step(x[0], x[0], w, x[0][:, None], x[0][:, None], None, None, None, torch.zeros(4, 8, 4))
    with pytest.raises(ValueError, match="CUDA"):
        L.block_norm_fwd(x)
    with pytest.raises(ValueError):
        L.short_conv_fwd(x[0], w)                                  # rows without cu_seqlens
    with pytest.raises(TypeError):
        L.short_conv_fwd(x[0], w, cu_seqlens=torch.tensor([0, 4]))  # int64


def test_column_ranges_do_not_overlap(L):
    """What the C side calls an overlap, on calls that end at a later check (no workspace)."""
    d = _conv(L, ld_x=32, ld_y=32, ld_dx=48)
    bwd = lambda at, d=d: _call(L, "kda_short_conv_bwd", 10, d, at=at)  # noqa: E731
    if torch.cuda.is_available():
        pytest.skip("made-up device addresses")
    assert bwd([(4, (1 << 28) + 32)]) == WORKSPACE            # x and dy side by side: both inputs anyway
    assert bwd([(6, (1 << 28) + 32)]) == ARG                  # dx in rows 48 apart over x in rows 32 apart
    e = _conv(L, ld_x=48, ld_y=48, ld_dx=48)
    assert bwd([(6, (1 << 28) + 32)], e) == WORKSPACE         # columns 16 .. 31 of rows of 48
    assert bwd([(6, (1 << 28) + 64)], e) == WORKSPACE         # 32 .. 47
    assert bwd([(6, (1 << 28) + 80)], e) == ARG               # 40 .. 55: over the next row's first
    assert bwd([(6, (1 << 28) - 32)], e) == WORKSPACE and bwd([(6, (1 << 28) - 16)], e) == ARG


def test_row_strides_of_views(L):
    c = L._Call.__new__(L._Call)
    c.dtype, c.device = torch.float32, -1
    t = torch.zeros(3, 5, 12)
    c.lead = (3, 5)
    assert c.rows(t, "t", (12,))[1] == 0
    assert c.rows(t[..., 4:8], "t", (4,))[1] == 12
    c.lead = (5,)
    assert c.rows(t[1, :, :4], "t", (4,))[1] == 12 and c.rows(t[1, :, :4].unflatten(-1, (2, 2)), "t", (2, 2))[1] == 12
    c.lead = (3,)
    assert c.rows(t[:, 2, :4], "t", (4,))[1] == 60
    c.lead = (3, 2)
    for bad in (t[:, 1:3, :4], t[:, :2].transpose(1, 2)[:, :2, :2].contiguous().transpose(1, 2)[:, :, :2]):
        with pytest.raises(ValueError):
            c.rows(bad, "t", tuple(bad.shape[2:]))
    c.lead = (4,)
    with pytest.raises(ValueError, match="overlap"):
        c.rows(torch.zeros(4).expand(4, 4), "t", (4,))
    with pytest.raises(ValueError, match="contiguous"):
        c.rows(torch.zeros(4, 8)[:, ::2], "t", (4,))
    with pytest.raises(TypeError):
        c.rows(torch.zeros(4, 4, dtype=torch.float64), "t", (4,))


def test_workspace_sizes(L):
    f = L._lib.kda_ssm_scan_fwd_workspace_bytes
    assert f(_ssm(L, B=256, D=12288), None) == 0          # enough sequences: no spans
    assert f(_ssm(L, N=5), None) == 0 and f(None, None) == 0
    b = L._lib.kda_ssm_scan_bwd_workspace_bytes
    assert b(_ssm(L, T=64), None) < b(_ssm(L, T=128), None) < b(_ssm(L, T=128, D=64), None)
    n = L._lib.kda_block_norm_bwd_workspace_bytes
    assert n(_norm(L), None) == 4 * 2 * 64 * 4 and n(_norm(L, rows=1 << 20), None) < 1 << 24
    assert ctypes.sizeof(L.kda_conv_dims) == 64 and ctypes.sizeof(L.kda_ssm_dims) == 88


# ------------------------------------------------------------------ index arithmetic that kernels and launchers share
def _host_program(tmp_path, body, header="kda_rows.cuh"):
    """Compiles `body` against a header of the kernels and runs it on the CPU; its output."""
    from gated_delta_rule_73_b200 import build as B
    src, exe = tmp_path / "p.cu", str(tmp_path / "p")
    src.write_text(f'#include <stdio.h>\n#include <stdlib.h>\n#include "{header}"\n'
                   f"using namespace kda;\nint main() {{\n{body}\nreturn 0;\n}}\n")
    subprocess.run([B._nvcc(), "-O1", "-std=c++17", *B.ARCH, "-I" + B.INC, "-I" + B.CSRC, str(src), "-o", exe], check=True,
                   capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120, cwd=os.fspath(tmp_path))
    assert r.returncode == 0, (r.returncode, r.stderr)
    return r.stdout.split()


def test_sequence_search_in_the_largest_tables(tmp_path):
    """Packed calls may have up to 2^31 - 1 sequences, nearly all of them empty: the search for a row's sequence
    and for a slot's reads inside the table at every size."""
    out = _host_program(tmp_path, """
    for (long long S : {3LL, (1LL << 30) + 5, (1LL << 31) - 1}) {
        int *cu = (int *)calloc(S + 1, sizeof(int));   // bounds of empty sequences; the pages stay untouched
        if (!cu) return 1;
        cu[S] = 100;
        const Seqs q{cu, (int)S, 100};
        const Span x = span_at(q, S - 1, 64), y = span_at(q, S, 64);   // 64 and 36 rows of the last sequence
        printf("%d %d %d %d %d %d %d\\n", q.at(0) == S - 1, q.at(99) == S - 1, x.seq == S - 1, (int)x.r0, x.n, (int)y.r0, y.n);
        free(cu);
    }""")
    assert out == 3 * ["1", "1", "1", "0", "64", "64", "36"]


def test_step_covers_the_most_sequences(tmp_path):
    """How the one-token scan divides sequences among parts: all of them once, up to the most that a call may have."""
    out = _host_program(tmp_path, """
    for (int S : {1, 2, 255, 2368, 2369, 0x7fffff00 - 2368, 0x7fffff00})
        for (int blocks : {1, 3, 384, 2368, 1 << 20}) {
            const StepParts x = step_parts(S, blocks);
            const bool all = (long long)x.count * x.per >= S && (long long)(x.count - 1) * x.per < S;
            printf("%d\\n", all && x.per > 0 && x.count > 0 && x.count <= 65535);
        }""", "kda_ssm.cuh")
    assert out == 35 * ["1"]
