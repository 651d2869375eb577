"""Host-side checks of the serving operators' C ABI that need no GPU: bad
arguments are refused before the device is touched, workspaces are sized."""
import ctypes as C
import os
import subprocess
import sys

import pytest
import torch

import verify_markov_head_gb300 as vm


@pytest.fixture(scope="module")
def host():
    return C.cast((C.c_float * 64)(), C.c_void_p)


def test_workspace_sizes():
    assert vm.dspark_cache_workspace_bytes(64, 32, 8, 128, 8) > 0
    assert vm.dspark_cache_workspace_bytes(64, 33, 8, 128, 8) == 0      # heads that do not divide
    assert vm.dspark_cache_workspace_bytes(64, 32, 8, 100, 8) == 0      # head size not a multiple of 8
    assert vm.dspark_cache_workspace_bytes(64, 32, 8, 264, 8) == 0
    assert vm.dspark_cache_workspace_bytes(4097, 32, 8, 128, 8) == 0
    assert vm.dspark_cache_workspace_bytes(64, 32, 8, 128, 18) == 0     # a block longer than gamma allows
    assert vm.dspark_logits_workspace_bytes(64, 8) >= 64 * 9 * 4
    assert vm.dspark_logits_workspace_bytes(64, 18) == 0
    assert vm.dspark_logits_workspace_bytes(0, 8) == 0


def test_plan_refuses_bad_sizes_and_host_memory(host):
    ok = dict(B=4, pages=100, width=8, page=16, T=32)

    def call(p=None, **kw):
        a = {**ok, **kw}
        return vm._lib.dspark_cache_plan(p, p, p, a["B"], p, p, a["pages"], p, a["width"], a["page"], p, p, p, p, p, p, p,
                                         a["T"], None, None)

    assert call(None) == -1 and call(host) == -1
    for kw in (dict(B=0), dict(B=4097), dict(pages=0), dict(page=0), dict(page=5000), dict(pages=1 << 28),
               dict(width=0), dict(width=1 << 28), dict(T=-1)):
        assert call(host, **kw) == -1, kw


def test_append_refuses_bad_arguments(host):
    def call(p, t=1, ks=256, vs=256, T=4, ps=4096, pages=10, page=16, heads=2, D=128):
        return vm._lib.dspark_cache_append(p, p, t, ks, vs, p, T, p, p, ps, pages, page, heads, D, None, None)

    assert call(None) == -1 and call(host) == -1
    assert call(host, t=2) == -4                                        # unknown type
    for kw in (dict(ks=255), dict(vs=260), dict(ks=128), dict(ps=4000), dict(D=12), dict(heads=0), dict(T=-1)):
        assert call(host, **kw) == -1, kw
    assert call(None, T=0) == 0                                         # nothing to write


def test_attention_refuses_bad_arguments(host):
    def call(p, qs=1024, t=1, ps=16384, page=16, width=4, B=2, N=4, Hq=8, Hkv=2, D=128, new=2, scale=1.0, ws=None, nb=0):
        return vm._lib.dspark_cache_attention(p, qs, p, p, t, ps, 10, page, p, width, p, p, p, B, N, Hq, Hkv, D, new,
                                              scale, p, None, ws, nb, None)

    assert call(None) == -1 and call(host) == -1
    assert call(host, t=5) == -4
    for kw in (dict(Hkv=3), dict(D=4), dict(new=0), dict(new=18), dict(scale=-1.0), dict(scale=float("inf")),
               dict(scale=float("nan")), dict(qs=1023), dict(qs=512), dict(ps=100), dict(B=0), dict(N=-1), dict(width=0)):
        assert call(host, **kw) == -1, kw
    assert call(None, N=0) == 0


@pytest.mark.parametrize("page,width,status", [(16, (1 << 27) - 16, 0), (16, (1 << 27) - 15, -1), (16, (1 << 27) - 1, -1),
                                               (1, (1 << 31) - 256, 0), (1, (1 << 31) - 255, -1), (1, (1 << 31) - 1, -1)])
def test_attention_refuses_tables_whose_positions_reach_the_end_of_32_bits(page, width, status):
    """The positions of the two steps behind a length stay below 2^31."""
    call = vm._lib.dspark_cache_attention
    assert call(None, 1024, None, None, 1, 16384, 10, page, None, width, None, None, None, 2, 0, 8, 2, 128, 2, 1.0, None, None,
                None, 0, None) == status


def test_logits_refuse_bad_arguments(host):
    def call(p, t=0, rs=64, B=2, R=3, V=64, hist=None, hist_len=None, draft=None, ds=0, nb=1 << 20,
             fill=float("-inf")):
        return vm._lib.dspark_logits_process(p, t, rs, p, B, R, V, hist, 4, hist_len, None, draft, ds, None, None, None,
                                             None, None, None, 0, None, fill, None, p, nb, None)

    assert call(None) == -1 and call(host) == -1
    assert call(host, t=3) == -4
    for kw in (dict(V=60), dict(V=0), dict(rs=63), dict(R=18), dict(R=0), dict(B=0), dict(B=70000), dict(nb=0),
               dict(fill=float("nan"))):
        assert call(host, **kw) == -1, kw


@pytest.mark.parametrize("heads,new", [(1, 1), (8, 1), (3, 3), (2, 8), (16, 1), (4, 8), (8, 8), (16, 8)])
def test_the_workspace_holds_two_tiles_of_rows_a_cta(heads, new):
    """Sums, maximum and weight of each row, for the tiles of either kernel, on 152 SMs."""
    rows = heads * new
    tile = max(8 if rows <= 8 else 32, min(128, 16 if rows <= 16 else 32 if rows <= 32 else 64 if rows <= 64 else 128))
    for D in (8, 64, 256):
        assert vm.dspark_cache_workspace_bytes(3, 2 * heads, 2, D, new) >= 256 + 152 * 32 + 2 * 152 * tile * (D + 2) * 4


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_draft_and_verification_import_without_the_serving_module():
    """Under another PyTorch than the module was built for: the package imports
    and the library answers; a serving operator says what is missing."""
    code = """
import torch
torch.__version__ = "0.0+other"
import verify_markov_head_gb300 as vm
assert vm.dspark_version() > 0 and vm.dspark_workspace_bytes(4, 7, 1024, 64) > 0
assert vm.dspark_cache_workspace_bytes(64, 32, 8, 128, 8) > 0
import inspect
inspect.getmembers(vm, inspect.isfunction)               # looking about in the package loads nothing
assert not hasattr(vm._serve, "__wrapped__")
for _ in range(2):
    try:
        vm.dspark_cache_append(None, None, None, None, None)
    except ImportError as e:
        assert "0.0+other" in str(e) and "build.py" in str(e), e
    else:
        raise AssertionError("no error")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_the_default_stream_of_a_call_is_the_current_one_by_pytorchs_public_function(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: type("S", (), {"cuda_stream": 1234}))
    assert vm._stream(None) == 1234
    assert vm._stream(77) == 77 and vm._stream(type("S", (), {"cuda_stream": 5})) == 5


@pytest.fixture
def builder(tmp_path, monkeypatch):
    """build.py with an output folder of its own and compilers that only write their output files."""
    from verify_markov_head_gb300 import build

    tool = tmp_path / "bin" / "nvcc"
    tool.parent.mkdir()
    tool.write_text(f"#!{sys.executable}\nimport sys\nopen(sys.argv[sys.argv.index('-o') + 1], 'w').write('made')\n")
    tool.chmod(0o755)
    (tool.parent / "g++").write_text(tool.read_text())
    (tool.parent / "g++").chmod(0o755)
    monkeypatch.setenv("NVCC", str(tool))
    monkeypatch.setenv("PATH", f"{tool.parent}{os.pathsep}{os.environ['PATH']}")
    monkeypatch.setattr(build, "OUT", str(tmp_path / "out"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "out" / "libdspark.so"))
    return build


def test_the_library_builds_without_pytorch(builder, monkeypatch):
    made = lambda: sorted(f for f in os.listdir(builder.OUT) if f.endswith(".so"))  # noqa: E731
    find = builder.importlib.util.find_spec
    monkeypatch.setattr(builder.importlib.util, "find_spec", lambda name: None if name == "torch" else find(name))
    assert builder.build() == builder.LIB
    assert made() == ["libdspark.so"]
    at = os.path.getmtime(builder.LIB)
    assert builder.build() == builder.LIB and os.path.getmtime(builder.LIB) == at     # nothing to do
    monkeypatch.setattr(builder.importlib.util, "find_spec", find)
    builder.build()                                              # PyTorch is there now: the module too
    assert made() == [f"_serve-{torch.__version__}.so", "libdspark.so"]


def test_the_library_stands_where_the_python_module_does_not_compile(builder, monkeypatch):
    def broken(cc):
        raise RuntimeError("g++ failed on serve_py.cpp")

    monkeypatch.setattr(builder, "_compile_serve", broken)
    with pytest.raises(RuntimeError, match="serve_py.cpp"):
        builder.build()
    assert os.listdir(builder.OUT).count("libdspark.so") == 1


def _plan_args(B=3, T=5):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return dict(seq_len=i(B), n_new=i(B), owned=i(B), ring=i(20), ring_state=i(2), block_table=i(B, 4), page_size=16,
                owned_out=i(B), ring_state_out=i(2), kv_len=i(B), q_off=i(B + 1), tile_off=i(B + 1), slot_map=i(T),
                positions=i(T))


def test_the_binding_names_what_is_wrong_with_a_tensor():
    a = _plan_args()
    with pytest.raises(vm.DsparkError):                          # all in order, but not on the device
        vm.dspark_cache_plan(**a, stream=0)
    for name in a:
        if name == "page_size":
            continue
        other = ("ring", "block_table")                          # any number of entries
        cases = [(a[name].float(), TypeError), (a[name].long(), TypeError), (None, TypeError), ([1, 2], TypeError)]
        if name not in other:
            cases += [(a[name][:-1], ValueError), (a[name][None], ValueError)]
        if name != "block_table":
            cases.append((torch.zeros(2 * a[name].numel(), dtype=torch.int32)[::2], ValueError))
        for bad, err in cases:
            # (slot_map's length is the number of slots, so positions is the one that differs)
            with pytest.raises(err, match="positions" if name == "slot_map" and err is ValueError and bad is not None and
                               bad.dim() == 1 and bad.is_contiguous() else name):
                vm.dspark_cache_plan(**{**a, name: bad}, stream=0)
    with pytest.raises(ValueError):
        vm.dspark_cache_plan(**{**a, "page_size": 1 << 40}, stream=0)
    with pytest.raises(TypeError):
        vm.dspark_cache_plan(**{**a, "page_size": "16"}, stream=0)
    with pytest.raises(AttributeError):
        vm.dspark_cache_plan(**a, stream="x")


@pytest.mark.parametrize("call", ["append", "attention"])
def test_the_binding_refuses_caches_that_do_not_fit(call):
    k = torch.zeros((6, 2, 16, 64), dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    x = torch.zeros((3, 2 if call == "append" else 4, 64), dtype=torch.bfloat16)
    ws = type("W", (), {"buf": torch.zeros(1 << 20, dtype=torch.uint8)})

    def run(k=k, v=k, x=x, y=None):
        y = torch.empty(x.shape, dtype=x.dtype) if y is None else y
        if call == "append":
            vm.dspark_cache_append(x, y, i(x.shape[0]), k, v, stream=0)
        else:
            vm.dspark_cache_attention(x, k, v, i(1, 4), i(1), i(2), i(2), y, ws, max_new=3, stream=0)

    with pytest.raises(vm.DsparkError):                          # all in order, but not on the device
        run()
    kv = torch.zeros((6, 2, 2, 16, 64), dtype=torch.bfloat16)    # keys and values of a page side by side: fits
    with pytest.raises(vm.DsparkError):
        run(k=kv[:, 0], v=kv[:, 1])
    for kw in (dict(v=k.float()), dict(v=k[:5]), dict(v=kv[:, 0]), dict(k=k.transpose(1, 2), v=k.transpose(1, 2)),
               dict(k=k[..., :32], v=k[..., :32]), dict(x=x[..., :32]), dict(x=x.float()), dict(x=x[:, :, None]),
               dict(x=torch.zeros((3, 64, x.shape[1]), dtype=torch.bfloat16).transpose(1, 2)), dict(y=x[:2])):
        with pytest.raises(ValueError):
            run(**kw)
    with pytest.raises(TypeError):
        run(k=k.double(), v=k.double())


def test_the_binding_refuses_logits_that_do_not_fit():
    x = torch.zeros((2, 3, 64))
    ws = type("W", (), {"buf": torch.zeros(1 << 16, dtype=torch.uint8)})
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    run = lambda x=x, out=None, **kw: vm.dspark_logits_process(  # noqa: E731
        x, torch.empty(x.shape, dtype=x.dtype) if out is None else out, ws, stream=0, **kw)
    good = dict(hist=i(2, 7), hist_len=i(2), prompt_len=i(2), draft_tok=i(2, 2), rep=torch.ones(2), freq=torch.ones(2),
                pres=torch.ones(2), bias_tok=i(4), bias_val=torch.zeros(4), bias_off=i(3), mask=i(2, 3, 2), live=i(2, 3))
    with pytest.raises(vm.DsparkError):                          # all in order, but not on the device
        run(**good)
    for kw in (dict(out=x[:1]), dict(out=x.double()), dict(x=torch.zeros((2, 64, 3)).transpose(1, 2)),
               dict(x=torch.zeros((2, 5, 64))[:, :3]), dict(hist=None), dict(hist_len=None), dict(hist=i(3, 7)),
               dict(draft_tok=i(2, 1)), dict(draft_tok=i(1, 2)), dict(bias_val=torch.zeros(3)), dict(bias_off=i(2)),
               dict(mask=i(2, 3, 3)), dict(live=i(3, 2)), dict(rep=torch.ones(3))):
        with pytest.raises(ValueError):
            run(**{**good, **kw})
    for kw in (dict(rep=torch.ones(2).double()), dict(mask=i(2, 3, 2).long()), dict(x=x.half()), dict(fill="low")):
        with pytest.raises(TypeError):
            run(**{**good, **kw})
