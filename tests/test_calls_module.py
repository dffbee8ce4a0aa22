"""The module of the speculation calls (``pa_calls.cpp``) on the host (no GPU): who needs it, when
it is built again, and what is built where it cannot be."""
import pytest
import torch


def cpu_pool():
    from paged_kv_cache_239_gb300.pool import BlockPool

    return BlockPool(4, 16, 1, 2, 64, tensor=torch.zeros((4, 2, 1, 2, 16, 64), dtype=torch.bfloat16))


def test_only_the_speculation_calls_need_the_module(pa_lib, monkeypatch):
    """Where the module cannot be loaded a pool does all that goes without it; the calls that
    need it say why they cannot."""
    def calls():
        raise RuntimeError("built for another torch")

    monkeypatch.setattr(pa_lib, "calls", calls)
    cache = cpu_pool()
    ids = [cache.allocate_block() for _ in range(4)]
    assert sorted(ids) == [0, 1, 2, 3] and cache.num_free() == 0
    cache.free_block(ids[0])
    cache.set_prefill_kernel("mma")
    assert cache.prefill_workspace_size(0, 0, 4, 4) == 0 and cache.tree_workspace_size(0, 0, 4, 4) == 0
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(RuntimeError, match="another torch"):
        cache.device_trim_sequences(i32(5), i32(2, 4), i32(2), i32(2))
    # and once it can be loaded, the same pool takes them
    monkeypatch.undo()
    with pytest.raises(ValueError, match="device"):
        cache.device_trim_sequences(i32(5), i32(2, 4), i32(2), i32(2))
    cache.close()


@pytest.fixture
def built(tmp_path, monkeypatch):
    """The build in a folder of its own, its compilers only taken down (they write their output)."""
    import subprocess

    from paged_kv_cache_239_gb300 import _build_lib as L

    for name in ("LIB_PATH", "CALLS_PATH"):
        monkeypatch.setattr(L, name, str(tmp_path / getattr(L, name).rsplit("/", 1)[1]))
    monkeypatch.setattr(L, "OUT_DIR", str(tmp_path))
    L.commands = []

    def run(cmd, **kw):
        L.commands.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(L.subprocess, "run", run)
    yield L
    del L.commands


def test_the_module_is_built_again_for_another_torch_or_python(built, monkeypatch):
    L = built
    assert L._stale()
    L.build()
    assert not L._stale() and len(L.commands) == len(L.SOURCES) + 3
    L.commands.clear()
    L.build()
    assert not L.commands
    # another torch on the disk (and in the next process), another Python: the module alone is built again
    def another(change):
        with pytest.MonkeyPatch.context() as m:
            change(m)
            assert L._stale()
            L.build()
            outs = [c[c.index("-o") + 1] for c in L.commands]
            assert len(outs) == 2 and outs[0].endswith("pa_calls.o") and "pagedcalls" in outs[1]
            assert not L._stale()
            L.commands.clear()
        assert L._stale()
        L.build()
        assert not L._stale()
        L.commands.clear()

    another(lambda m: (m.setattr(L, "_installed_torch", lambda: "9.9.0"), m.setattr(torch, "__version__", "9.9.0")))
    another(lambda m: m.setattr(L, "_python_abi", lambda: "cpython-399-other"))
    # another torch in this process than the one on the disk
    monkeypatch.setattr(torch, "__version__", "9.9.1")
    assert L._stale()


def test_another_torchs_module_is_not_loaded(pa_lib, monkeypatch):
    """Refused before any of its code is linked, and with what mends it."""
    import importlib.util

    assert pa_lib.calls() is not None
    monkeypatch.setattr(pa_lib, "_calls", None)
    monkeypatch.setattr(importlib.util, "module_from_spec", lambda spec: pytest.fail("loaded"))
    monkeypatch.setattr(torch, "__version__", "9.9.0")
    with pytest.raises(RuntimeError, match="9.9.0.*_build_lib"):
        pa_lib.calls()
    monkeypatch.setattr(torch, "__version__", torch.version.__version__)
    monkeypatch.setattr(pa_lib._build_lib, "_python_abi", lambda: "cpython-399-other")
    with pytest.raises(RuntimeError, match="cpython-399-other.*_build_lib"):
        pa_lib.calls()


@pytest.mark.parametrize("what", ["no torch", "no c10 for CUDA", "no Python headers"])
def test_the_library_is_built_where_the_module_cannot_be(built, monkeypatch, tmp_path, what):
    """C programs need neither torch nor Python's headers."""
    L = built
    if what == "no torch":
        find = L.importlib.util.find_spec
        monkeypatch.setattr(L.importlib.util, "find_spec", lambda name: None if name == "torch" else find(name))
    elif what == "no c10 for CUDA":
        (tmp_path / "torch").mkdir()
        monkeypatch.setattr(L, "_torch_dir", lambda: str(tmp_path / "torch"))
    else:
        monkeypatch.setattr(L.sysconfig, "get_paths", lambda: {"include": str(tmp_path / "none")})
    assert L.build() == L.LIB_PATH and L.os.path.exists(L.LIB_PATH)
    assert len(L.commands) == len(L.SOURCES) + 1 and not L.os.path.exists(L.CALLS_PATH)
    L.commands.clear()
    L.build()
    assert not L.commands   # (nothing is stale)


def test_a_module_that_does_not_compile_fails_the_build_after_the_library(built, monkeypatch):
    L = built
    run = L.subprocess.run

    def fail(cmd, **kw):
        done = run(cmd, **kw)
        if cmd[0] == "g++":
            done.returncode, done.stderr = 1, "no such header"
        return done

    monkeypatch.setattr(L.subprocess, "run", fail)
    with pytest.raises(RuntimeError, match="pa_calls.cpp"):
        L.build()
    assert not L._library_stale() and L._calls_stale()


def test_a_build_for_the_same_torch_leaves_the_stamp_in_its_place(built, monkeypatch):
    """Processes that build at once do not take the module from one another."""
    L = built
    L.build()
    stamp = L.read_calls_stamp()
    seen = []
    replace = L.os.replace

    def watched(a, b):
        replace(a, b)
        seen.append(L.read_calls_stamp())

    monkeypatch.setattr(L.os, "replace", watched)
    monkeypatch.setattr(L.os, "remove", lambda path: pytest.fail("removed"))
    L.build(force=True)
    assert seen and all(x == stamp for x in seen)
