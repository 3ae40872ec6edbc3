"""The serving calls' argument checks and layouts, without a device."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 4
P = 4096            # an aligned address that is never used


@pytest.fixture(scope="module")
def lib():
    from exact_io_aware_100_b200 import build, load_library
    build.build()
    return load_library()


def rotary_layout(**over):
    import exact_io_aware_100_b200 as fa
    v = dict(B=2, H=4, H_kv=2, N=8, d=64, rotary_dim=64, interleaved=0, positions_batch=0)
    for n, h in (("q", 4), ("k", 2), ("q_out", 4), ("k_out", 2)):
        v |= {n + "_batch": h * 8 * 64, n + "_head": 8 * 64, n + "_row": 64}
    return fa.FaRotaryLayout(**(v | over))


def paged_layout(**over):
    import exact_io_aware_100_b200 as fa
    v = dict(B=2, H=4, H_kv=2, d=64, N=1, num_pages=10, page_size=16, max_pages=4, table_stride=4, cu_seqlens=None, total=0,
             rotary_dim=64, interleaved=0)
    for n, h, rows in (("q", 4, 1), ("o", 4, 1), ("k", 2, 1), ("v", 2, 1), ("k_pages", 2, 16), ("v_pages", 2, 16)):
        v |= {n + "_batch": h * rows * 64, n + "_head": rows * 64, n + "_row": 64}
    return fa.FaPagedLayout(**(v | over))


def pages_layout(**over):
    import exact_io_aware_100_b200 as fa
    return fa.FaPagesLayout(**(dict(num_seqs=3, num_pages=10, page_size=16, max_pages=4, table_stride=4) | over))


def test_structs_match_the_header(tmp_path):
    import exact_io_aware_100_b200 as fa
    want = [("fa_rotary_layout", fa.FaRotaryLayout, ["positions_batch", "q", "k_out"], ["positions_batch", "q_batch", "k_out_batch"]),
            ("fa_paged_layout", fa.FaPagedLayout, ["table_stride", "q", "v_pages", "cu_seqlens", "interleaved"],
             ["table_stride", "q_batch", "v_pages_batch", "cu_seqlens", "interleaved"]),
            ("fa_pages_layout", fa.FaPagesLayout, ["max_pages", "table_stride"], ["max_pages", "table_stride"])]
    body = "".join('printf("%%zu\\n", sizeof(%s));' % c + "".join('printf("%%zu\\n", offsetof(%s, %s));' % (c, f) for f in fs)
                   for c, _, fs, _ in want)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "fa.h"\nint main(void) { %s return 0; }\n' % body)
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(tmp_path / "l"), str(src)], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [x for _, t, _, fs in want for x in [ctypes.sizeof(t)] + [getattr(t, f).offset for f in fs]]


@pytest.mark.parametrize("over,code", [
    (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(H_kv=-1), INVALID), (dict(N=-1), INVALID), (dict(d=0), INVALID),
    (dict(d=1025), INVALID), (dict(rotary_dim=63), INVALID), (dict(rotary_dim=66), INVALID), (dict(rotary_dim=-2), INVALID),
    (dict(H=1 << 16), INVALID), (dict(H_kv=1 << 16), INVALID),
    (dict(B=1 << 20, N=1 << 12), INVALID), (dict(q_out_row=0), INVALID), (dict(k_out_head=-64), INVALID), (dict(N=0), OK),
])
def test_rotary_refuses(lib, over, code):
    assert lib.fa_rotary(P, P, P, P, None, P, rotary_layout(**over), 1.0, 0, 0, None) == code


def test_rotary_refuses_pointers_types_and_magnitude(lib):
    L, f = rotary_layout(), lib.fa_rotary
    assert f(P, P, P, P, None, P, None, 1.0, 0, 0, None) == INVALID
    assert f(P, P, P, P, None, P, L, 1.0, 0, 7, None) == UNSUPPORTED
    assert f(P, P, P, P, None, P, L, float("nan"), 0, 0, None) == INVALID
    assert f(None, P, P, P, None, P, L, 1.0, 0, 0, None) == ALIGN
    assert f(P, None, P, P, None, P, L, 1.0, 0, 0, None) == ALIGN
    assert f(P, P, P + 1, P, None, P, L, 1.0, 0, 0, None) == ALIGN
    assert f(P + 2, P, P, P, None, P, L, 1.0, 0, 1, None) == ALIGN               # float32 wants 4 bytes
    assert f(P, P, P, P, P + 2, P, L, 1.0, 0, 0, None) == ALIGN
    assert f(P, P, P, P, None, P + 4, L, 1.0, 0, 0, None) == ALIGN
    assert f(P, P, P, P, None, None, L, 1.0, 0, 0, None) == ALIGN
    # nothing to turn: no frequencies wanted; no rows: nothing launched
    assert f(P, None, P, None, None, None, rotary_layout(H_kv=0, N=0, rotary_dim=0), 1.0, 0, 0, None) == OK


CACHE = [
    (dict(B=0), INVALID), (dict(H_kv=0), INVALID), (dict(num_pages=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(page_size=12), INVALID), (dict(page_size=0), INVALID), (dict(page_size=65544), INVALID),
    (dict(max_pages=1 << 28), INVALID), (dict(max_pages=(1 << 26) + 1, table_stride=1 << 27), INVALID),
    (dict(table_stride=3), INVALID), (dict(k_pages_row=60), ALIGN),
    (dict(v_pages_head=0), ALIGN), (dict(k_pages_batch=-64), ALIGN),
]


@pytest.mark.parametrize("over,code", CACHE + [
    (dict(N=-1), INVALID), (dict(rotary_dim=63), INVALID), (dict(rotary_dim=128), INVALID), (dict(q_head=68), ALIGN),
    (dict(k_batch=4), ALIGN), (dict(cu_seqlens=P + 2, total=4), ALIGN), (dict(cu_seqlens=P, total=-1), INVALID),
    (dict(H=0), INVALID), (dict(N=0), OK), (dict(cu_seqlens=P, total=0), OK),
])
def test_append_refuses(lib, over, code):
    assert lib.fa_paged_append(P, P, P, P, P, P, P, P, P, paged_layout(**over), 1.0, None) == code


def test_append_refuses_pointers(lib):
    L, f = paged_layout(), lib.fa_paged_append
    args = [P] * 9
    assert f(*args, None, 1.0, None) == INVALID
    assert f(*args, L, float("inf"), None) == INVALID
    for at in range(1, 8):
        bad = list(args)
        bad[at] = None
        assert f(*bad, L, 1.0, None) == ALIGN
    assert f(P, P, P, P, P + 8, P, P, P, P, L, 1.0, None) == ALIGN
    assert f(P, P, P, P, P, P, P, P, P + 4, L, 1.0, None) == ALIGN


@pytest.mark.parametrize("over,code", CACHE + [
    (dict(N=0), INVALID), (dict(H=5), INVALID), (dict(H=0), INVALID), (dict(q_head=68), ALIGN), (dict(o_batch=0), ALIGN),
    (dict(B=1 << 20, H=1 << 12), INVALID), (dict(B=1, N=1 << 18), INVALID),
])
def test_decode_refuses(lib, over, code):
    L = paged_layout(**over)
    assert lib.fa_paged_decode(P, P, P, P, P, P, P, L, 0.1, 1, P, 1 << 40, None) == code
    assert lib.fa_paged_decode_workspace_size(L) == 0


def test_decode_refuses_pointers_scale_and_workspace(lib):
    L, f = paged_layout(), lib.fa_paged_decode
    need = lib.fa_paged_decode_workspace_size(L)
    assert need > 0 and lib.fa_paged_decode_workspace_size(None) == 0
    args = [P] * 7
    assert f(*args, None, 0.1, 1, P, need, None) == INVALID
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert f(*args, L, scale, 1, P, need, None) == INVALID
    for at in range(7):
        bad = list(args)
        bad[at] = None
        assert f(*bad, L, 0.1, 1, P, need, None) == ALIGN
    assert f(*args, L, 0.1, 1, None, 0, None) == WORKSPACE
    assert f(*args, L, 0.1, 1, P, need - 1, None) == WORKSPACE
    assert f(*args, L, 0.1, 1, P + 16, need, None) == WORKSPACE


@pytest.mark.parametrize("over", [dict(num_seqs=0), dict(num_pages=0), dict(page_size=0), dict(max_pages=0),
                                  dict(table_stride=3), dict(page_size=1 << 30), dict(num_pages=1 << 30)])
def test_page_calls_refuse_layouts(lib, over):
    L, big = pages_layout(**over), 1 << 40
    assert lib.fa_pages_extend(P, P, P, L, P, P, 2, P, P, big, None) == INVALID
    assert lib.fa_pages_fork(P, P, P, L, P, P, 2, P, P, P, big, None) == INVALID
    assert lib.fa_pages_free(P, P, P, L, P, 2, None) == INVALID
    assert lib.fa_pages_compact(P, P, P, L, P, P, big, None) == INVALID
    assert lib.fa_pages_workspace_size(L, 2) == 0


def test_page_calls_refuse_arguments(lib):
    L = pages_layout()
    need = lib.fa_pages_workspace_size(L, 2)
    assert need > 0 and lib.fa_pages_workspace_size(None, 2) == 0 and lib.fa_pages_workspace_size(L, -1) == 0
    e, k = lib.fa_pages_extend, lib.fa_pages_fork
    assert e(P, P, P, L, P, P, -1, P, P, need, None) == INVALID
    assert e(P, P, P, L, None, P, 2, P, P, need, None) == ALIGN
    assert e(P, P, P, L, P, P, 2, None, P, need, None) == ALIGN
    assert e(None, P, P, L, P, P, 2, P, P, need, None) == ALIGN
    assert e(P, P, P, L, P, P, 2, P, P, need - 1, None) == WORKSPACE
    assert e(P, P, P, L, P, P, 2, P, None, need, None) == WORKSPACE
    assert k(P, P, P, L, P, P, 2, None, P, P, need, None) == ALIGN
    assert k(P, P, P, L, P, P, 2, P, P, P + 4, need, None) == WORKSPACE
    assert lib.fa_pages_free(P, P, P, L, P + 2, 2, None) == ALIGN
    assert lib.fa_pages_compact(P, P, P, L, None, P, need, None) == ALIGN
    assert lib.fa_pages_compact(P, P, P, L, P, None, 0, None) == WORKSPACE
    c, C = lib.fa_pages_copy, paged_layout()
    assert c(P, P, P, 2, None, None) == INVALID
    assert c(P, P, P, -1, C, None) == INVALID
    assert c(P, P, P, 0, C, None) == OK
    assert c(P, P, None, 2, C, None) == ALIGN
    assert c(P + 8, P, P, 2, C, None) == ALIGN
    assert c(P, P, P, 2, paged_layout(d=60), None) == INVALID
    assert c(P, P, P, 2, paged_layout(k_pages_row=4), None) == ALIGN


def test_binding_refuses(lib):
    import torch
    import exact_io_aware_100_b200 as fa
    q = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    f = torch.zeros(32, dtype=torch.float64)
    pages, table, lens = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.rotary(q, None, f)
    with pytest.raises(ValueError, match="dtype"):
        fa.rotary(q.half(), None, f)
    with pytest.raises(ValueError, match="freqs"):
        fa.rotary(q, None, f.float())
    with pytest.raises(ValueError, match="positions"):
        fa.rotary(q, None, f, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="int32"):
        fa.rotary(q, None, f, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="agree"):
        fa.rotary(q, torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16), f)
    with pytest.raises(ValueError, match="CUDA"):
        fa.paged_decode(q, pages, pages, table, lens)
    with pytest.raises(ValueError, match="agree"):
        fa.paged_decode(q, pages, pages, table, torch.ones(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="k_pages"):
        fa.paged_decode(q, pages.float(), pages, table, lens)
    with pytest.raises(ValueError, match="heads"):
        fa.paged_append(q[:, :1], q[:, :1], pages, pages, table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        fa.pages_free(table, lens, lens, 16, lens)
    with pytest.raises(ValueError, match="length"):
        fa.pages_extend(table, lens, lens, 16, lens, torch.ones(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="copies"):
        fa.pages_copy(pages, pages, torch.zeros(2, 2, dtype=torch.int32))


def test_frequencies(lib):
    import math
    import exact_io_aware_100_b200 as fa
    f, m = fa.rotary_frequencies(8, 10000.0, device="cpu")
    assert m == 1.0 and f.tolist() == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-15)
    assert fa.rotary_frequencies(8, 10000.0, "linear", 4.0, device="cpu")[0].tolist() == pytest.approx([0.25, 0.025, 0.0025, 0.00025])
    g = fa.rotary_frequencies(8, 10000.0, "ntk", 4.0, device="cpu")[0].tolist()
    assert g[0] == 1.0 and g[3] == pytest.approx(0.001 / 4)
    # turns over 1000 positions: 159, 15.9, 1.59, 0.159
    g = fa.rotary_frequencies(8, 10000.0, "bands", 4.0, 1000, device="cpu")[0].tolist()
    keep = (10 / (2 * math.pi) - 1) / 3
    assert g == pytest.approx([1.0, 0.1, 0.01 * keep + 0.0025 * (1 - keep), 0.00025])
    # pair index of 32 turns 0.70 -> 0, of one turn 2.20 -> 3: the ramp runs over pairs 0 to 3
    g, m = fa.rotary_frequencies(8, 10000.0, "yarn", 4.0, 1000, device="cpu")
    assert m == pytest.approx(0.1 * math.log(4.0) + 1.0)
    assert g.tolist() == pytest.approx([f0 * (1 - i / 3) + f0 / 4 * (i / 3) for i, f0 in enumerate([1.0, 0.1, 0.01, 0.001])])
    assert fa.rotary_frequencies(0, device="cpu")[0].numel() == 0
    for bad in (dict(scaling="x"), dict(scaling="yarn", factor=2.0), dict(base=-1.0), dict(factor=0.5, scaling="linear"),
                dict(scaling="bands", original_length=100, low=4.0, high=1.0)):
        with pytest.raises(ValueError):
            fa.rotary_frequencies(8, **({"device": "cpu"} | bad))
    with pytest.raises(ValueError):
        fa.rotary_frequencies(7, device="cpu")
