"""Refusals of the serving operators (no GPU): every argument the host can
see is checked before the device is touched, so made-up pointers are never
followed."""
import ctypes as C
import math

import pytest

mk = pytest.importorskip("persistent_decode_megakernel_02_b200.mk")
lib = mk._lib
A = 1 << 20          # an aligned made-up address


def cache(**kw):
    f = dict(k=A, v=A, page_table=A, n_seqs=2, pages_per_seq=4, num_pages=8, page_size=16, n_kv_heads=2,
             head_dim=64, dtype=mk.MK_BF16)
    f.update(kw)
    return mk.PagedKVStruct(**f)


BAD_CACHES = [dict(k=None), dict(v=A + 8), dict(page_table=None), dict(page_table=A + 2), dict(n_seqs=0),
              dict(pages_per_seq=0), dict(num_pages=0), dict(page_size=0), dict(page_size=-1), dict(n_kv_heads=0),
              dict(head_dim=96), dict(head_dim=0), dict(dtype=2), dict(dtype=-1),
              dict(pages_per_seq=1 << 20, page_size=1 << 20),
              dict(num_pages=1 << 26)]


def append(c=None, **kw):
    a = dict(cu=A, start=A, n=4, nq=4, q=A, qs=256, k=A, ks=128, v=A, vs=128, theta=1e4, qo=A, qos=256, ko=None,
             kos=0, status=None)
    a.update(kw)
    c = cache() if c is None else c
    return lib.mk_kv_append(C.byref(c), a["cu"], a["start"], a["n"], a["nq"], a["q"], a["qs"], a["k"], a["ks"],
                            a["v"], a["vs"], a["theta"], a["qo"], a["qos"], a["ko"], a["kos"], a["status"], None)


def paged(c=None, **kw):
    a = dict(lens=A, max_len=64, nq=4, q=A, qs=256, scale=0.125, out=A, os=256, ws=A, wsb=1 << 40, status=None)
    a.update(kw)
    c = cache() if c is None else c
    return lib.mk_paged_attention(C.byref(c), a["lens"], a["max_len"], a["nq"], a["q"], a["qs"], a["scale"],
                                  a["out"], a["os"], a["ws"], a["wsb"], a["status"], None)


def prompt(**kw):
    a = dict(dtype=mk.MK_FP16, nq=4, nkv=2, d=64, cu=A, ns=2, n=10, max_len=8, q=A, qs=256, k=A, ks=128, v=A,
             vs=128, scale=0.125, out=A, os=256, status=None)
    a.update(kw)
    return lib.mk_prompt_attention(a["dtype"], a["nq"], a["nkv"], a["d"], a["cu"], a["ns"], a["n"], a["max_len"],
                                   a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["scale"], a["out"], a["os"],
                                   a["status"], None)


def sample(**kw):
    a = dict(logits=A, stride=100, rows=2, vocab=100, u=A, t=A, k=A, p=A, m=A, out=A)
    a.update(kw)
    return lib.mk_sample(a["logits"], a["stride"], a["rows"], a["vocab"], a["u"], a["t"], a["k"], a["p"], a["m"],
                         a["out"], None)


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_caches_are_checked(bad):
    assert append(cache(**bad)) == mk.MK_ERR_INVALID
    assert paged(cache(**bad)) == mk.MK_ERR_INVALID


@pytest.mark.parametrize("bad", [
    dict(cu=None), dict(cu=A + 1), dict(start=None), dict(n=-1), dict(nq=3), dict(nq=18), dict(nq=-2),
    dict(q=None), dict(q=A + 2), dict(qs=248), dict(qs=260), dict(qs=0), dict(k=None), dict(ks=120), dict(ks=132),
    dict(v=A + 8), dict(vs=64), dict(theta=1.0), dict(theta=math.nan), dict(theta=math.inf), dict(qo=None),
    dict(qos=128), dict(ko=A + 4, kos=128), dict(ko=A, kos=64), dict(nq=0), dict(nq=0, q=None),
    dict(q=A, qo=A, qs=256, qos=512), dict(ko=A, kos=256), dict(status=A + 2)], ids=str)
def test_append_refusals(bad):
    assert append(**bad) == mk.MK_ERR_INVALID


@pytest.mark.parametrize("bad", [
    dict(lens=None), dict(lens=A + 2), dict(max_len=-1), dict(max_len=65), dict(nq=3), dict(nq=0), dict(nq=18),
    dict(q=None), dict(q=A + 8), dict(qs=128), dict(qs=257), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=math.nan), dict(scale=math.inf), dict(out=None), dict(os=8), dict(ws=A + 8), dict(status=A + 1)],
    ids=str)
def test_paged_refusals(bad):
    assert paged(**bad) == mk.MK_ERR_INVALID


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(nq=5), dict(nq=0), dict(nkv=0), dict(nq=18), dict(d=80), dict(d=256), dict(cu=None),
    dict(cu=A + 2), dict(ns=0), dict(n=-1), dict(n=(1 << 31) - 1), dict(ns=1 << 29, nq=8, nkv=4, n=1, qs=512, os=512, ks=256, vs=256), dict(max_len=-1), dict(q=None), dict(qs=255), dict(qs=0), dict(k=A + 2),
    dict(ks=64), dict(v=None), dict(vs=129), dict(scale=0.0), dict(scale=math.nan), dict(out=None), dict(os=192),
    dict(status=A + 3)], ids=str)
def test_prompt_refusals(bad):
    assert prompt(**bad) == mk.MK_ERR_INVALID


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(logits=A + 2), dict(stride=99), dict(rows=-1), dict(rows=(1 << 24) + 1), dict(vocab=0), dict(u=None),
    dict(vocab=mk.MAX_VOCAB + 1, stride=1 << 21), dict(out=None), dict(out=A + 1), dict(t=A + 2), dict(k=A + 1),
    dict(p=A + 3), dict(m=A + 2)], ids=str)
def test_sample_refusals(bad):
    assert sample(**bad) == mk.MK_ERR_INVALID


def test_workspace_refusals():
    n = C.c_size_t(7)
    ask = lambda c, m, nq: lib.mk_paged_attention_workspace(C.byref(c), m, nq, C.byref(n))
    for c, m, nq in ((cache(head_dim=32), 10, 4), (cache(num_pages=1 << 30), 10, 4), (cache(), 65, 4), (cache(), -1, 4), (cache(), 10, 5),
                     (cache(), 10, 0)):
        assert ask(c, m, nq) == mk.MK_ERR_INVALID and n.value == 0
    assert lib.mk_paged_attention_workspace(None, 1, 1, C.byref(n)) == mk.MK_ERR_INVALID
    assert lib.mk_paged_attention_workspace(C.byref(cache()), 1, 4, None) == mk.MK_ERR_INVALID


def test_paged_work_that_does_not_fit_an_int():
    # shared pages can make a batch longer than any device's memory
    c = cache(n_seqs=1 << 20, pages_per_seq=1 << 16, n_kv_heads=8)
    assert paged(c, nq=8, q=A, qs=512, os=512, max_len=1 << 20) == mk.MK_ERR_INVALID


def test_nothing_to_do_touches_no_device():
    assert append(n=0) == mk.MK_OK
    assert prompt(n=0) == mk.MK_OK
    assert sample(rows=0) == mk.MK_OK


def test_null_cache():
    assert lib.mk_kv_append(None, A, A, 1, 0, None, 0, A, 128, A, 128, 1e4, None, 0, None, 0, None, None) \
        == mk.MK_ERR_INVALID
    assert lib.mk_paged_attention(None, A, 1, 4, A, 256, 1.0, A, 256, A, 1 << 30, None, None) == mk.MK_ERR_INVALID


def test_cache_struct_matches_the_c_compiler(tmp_path):
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    lines = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{mk.HEADER_PATH}"', "int main(void) {",
             'printf("%zu\\n", sizeof(mk_paged_kv));']
    names = [n for n, _ in mk.PagedKVStruct._fields_]
    lines += [f'printf("%zu\\n", offsetof(mk_paged_kv, {n}));' for n in names]
    lines += ['printf("%d\\n", MK_MAX_GROUP);', 'printf("%d\\n", MK_MAX_VOCAB);', "return 0;", "}"]
    src, exe = tmp_path / "t.c", tmp_path / "t"
    src.write_text("\n".join(lines))
    subprocess.check_call(["gcc", "-std=c11", "-o", str(exe), str(src)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    want = [C.sizeof(mk.PagedKVStruct)] + [getattr(mk.PagedKVStruct, n).offset for n in names]
    assert got == want + [mk.MAX_GROUP, mk.MAX_VOCAB]


@pytest.mark.parametrize("n", [1 << 31, (1 << 32) + 5, -(1 << 31) - 1, 1.0, None, "4"])
def test_binding_numbers_that_are_no_int(n):
    with pytest.raises(mk.MkError) as e:      # ctypes alone would make 5 of the second
        mk._ints("call", fine=(1 << 31) - 1, max_len=n)
    assert e.value.status == mk.MK_ERR_INVALID and "max_len" in str(e.value)


def test_binding_checks_its_tensors():
    import torch
    k = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(mk.MkError) as e:      # not on a GPU
        mk.PagedKV(k, k, torch.zeros(1, 2, dtype=torch.int32))
    assert e.value.status == mk.MK_ERR_INVALID
    with pytest.raises(mk.MkError):
        mk.sample(torch.zeros(1, 8), torch.zeros(1), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(mk.MkError):
        mk.prompt_attention(k[0], k[0], k[0], torch.zeros(2, dtype=torch.int32), 4, k[0])


def one_row_layouts():
    """[1][8][64] views whose heads are not contiguous."""
    import torch
    x = torch.zeros(1, 8, 3, 64, dtype=torch.bfloat16)
    return {"interleaved": x[:, :, 1], "transposed": torch.zeros(1, 64, 8, dtype=torch.bfloat16).transpose(1, 2),
            "sliced": torch.zeros(1, 8, 128, dtype=torch.bfloat16)[..., :64],
            "every second": torch.zeros(1, 8, 128, dtype=torch.bfloat16)[..., ::2],
            "expanded heads": torch.zeros(1, 1, 64, dtype=torch.bfloat16).expand(1, 8, 64),
            "expanded elements": torch.zeros(1, 8, 1, dtype=torch.bfloat16).expand(1, 8, 64)}


@pytest.mark.parametrize("name", list(one_row_layouts()))
def test_a_single_row_has_contiguous_heads_too(name):
    t = one_row_layouts()[name]
    with pytest.raises(mk.MkError) as e:      # -1 is a CPU tensor's device number
        mk._rows("call", "q", t, t.dtype, -1, (1, 8, 64))
    assert e.value.status == mk.MK_ERR_INVALID
    assert mk._row_stride(t) < 0              # the rule itself, which the compiled way asks too


def test_layouts_that_are_taken():
    import torch
    x = torch.zeros(5, 12, 64)
    rows = lambda t: mk._rows("call", "q", t, t.dtype, -1, tuple(t.shape))
    assert rows(x) == 12 * 64 and rows(x[:, 2:6]) == 12 * 64 and rows(x[::2, :3]) == 2 * 12 * 64
    # of one row the row stride does not matter, of one head the head stride, of none anything
    assert rows(x[:1, 2:6]) == 4 * 64 and rows(x.as_strided((1, 12, 64), (7, 64, 1))) == 12 * 64
    assert rows(x[:, ::12]) == 12 * 64 and rows(x[:0].transpose(1, 2)) == 12 * 64


def test_the_prompt_guard_s_warps_share_no_column(tmp_path):
    """Two warps take values that are not finite out of a tile and remember them per column; if a
    column belonged to both, one could wait for the other for good."""
    import os
    import subprocess
    here, exe = os.path.dirname(os.path.abspath(__file__)), str(tmp_path / "guard_check")
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-I/usr/local/cuda/include", os.path.join(here, "guard_check.cpp"), "-o", exe])
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout


def test_the_serving_operators_wait_at_no_barrier_a_warp_may_miss():
    """Named barriers have no bound: none is left where a role may give up alone."""
    import os
    import re
    csrc = os.path.join(os.path.dirname(mk.LIB_PATH), "csrc")
    for name in ("mk_prompt_attn.cu", "mk_tc.cuh", "mk_ops.cuh"):
        with open(os.path.join(csrc, name)) as f:
            assert not re.search(r"\bbar(rier)?\.(cta\.)?(sync|red|arrive)", f.read()), name


def compiler_log(**registers):
    lines = []
    for name, n in registers.items():
        lines += [f"ptxas info    : Compiling entry function '_ZN2mk50_GLOBAL__N__92e1c366{name}INS_4Fp16ELi64EEEv' for 'sm_100a'",
                  f"ptxas info    : Function properties for _ZN2mk50_GLOBAL__N__92e1c366{name}INS_4Fp16ELi64EEEv",
                  "    8 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads", f"ptxas info    : Used {n} registers, used 1 barriers"]
    return "\n".join(lines)


def test_a_build_with_other_launch_registers_stops():
    """Kernels that split their registers are refused at run time with any other number."""
    from persistent_decode_megakernel_02_b200 import build as b
    good = dict(mk_step_kernel=168, repack_rows_kernel=30, prompt_attn_kernel=168)
    b.check_registers(compiler_log(**good))
    for name in ("mk_step_kernel", "prompt_attn_kernel"):
        with pytest.raises(RuntimeError, match=f"{name}.*160 registers"):
            b.check_registers(compiler_log(**{**good, name: 160}))
        with pytest.raises(RuntimeError, match=f"no registers for {name}"):
            b.check_registers(compiler_log(**{k: v for k, v in good.items() if k != name}))


def test_the_build_s_launch_registers_are_the_sources():
    import os
    import re
    from persistent_decode_megakernel_02_b200 import build as b
    text = "".join(open(os.path.join(b.CSRC, f)).read() for f in ("mk_internal.h", "mk_prompt_attn.cu"))
    assert dict(re.findall(r"constexpr int (kLaunchRegs\w*) = (\d+)", text)) == {"kLaunchRegs": "168", "kLaunchRegsPrompt": "168"}
    assert set(b.LAUNCH_REGISTERS.values()) == {168}


def test_outputs_over_inputs_that_are_still_read():
    """Rows may be rotated in place; an output over another operand is refused, as far as the first
    elements show it."""
    own = dict(q=A, k=2 * A, v=3 * A, qo=4 * A, ko=5 * A, kos=128)
    for bad in (dict(qo=2 * A), dict(qo=3 * A), dict(ko=3 * A), dict(ko=A), dict(ko=4 * A), dict(k=A, qo=A), dict(v=A, qo=A),
                dict(v=2 * A, ko=2 * A)):
        assert append(**{**own, **bad}) == mk.MK_ERR_INVALID, bad
    for bad in (dict(out=2 * A), dict(out=3 * A)):
        assert prompt(**{**dict(q=A, k=2 * A, v=3 * A, out=4 * A, os=256), **bad}) == mk.MK_ERR_INVALID, bad
    assert paged(q=A, out=A, qs=256, os=512) == mk.MK_ERR_INVALID


@pytest.mark.skipif(__import__("torch").cuda.is_available(), reason="made-up pointers")
def test_the_forms_in_place_pass_the_checks():
    # without a device the next thing a call meets is its absence
    own = dict(q=A, k=2 * A, v=3 * A, qo=4 * A, ko=5 * A, kos=128)
    for ok in (dict(), dict(qo=A), dict(ko=2 * A), dict(qo=A, ko=2 * A), dict(ko=None), dict(nq=0, q=None, qo=None),
               dict(nq=0, q=None, qo=None, ko=2 * A)):
        assert append(**{**own, **ok}) == mk.MK_ERR_CUDA, ok
    assert prompt(q=A, k=2 * A, v=3 * A, out=4 * A) == mk.MK_ERR_CUDA
    assert paged(q=A, out=A) == mk.MK_ERR_CUDA
