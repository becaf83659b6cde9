"""Loading of the library and of the marshalling module, on the CPU: a module that is missing or does not load is
named by every call that needs it, and by no other; threads that come first at once all get a complete one."""
import threading

import pytest
import torch


@pytest.fixture
def pk(monkeypatch):
    from paged_kv_cache_10_gb300 import build, pagedkv
    build.build()
    monkeypatch.setattr(pagedkv, "_lib", None)
    monkeypatch.setattr(pagedkv, "_native", None)
    return pagedkv


def append(pk):
    d = pk.CacheDesc(num_blocks=1, num_kv_heads=1, head_size=64)
    z = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    pk.paged_kv_append(z, z, torch.zeros(1, dtype=torch.int64), z, z, d)


def test_a_missing_module_is_named_every_time(pk, monkeypatch, tmp_path):
    path = pk.BINDING_PATH
    monkeypatch.setattr(pk, "BINDING_PATH", str(tmp_path / "none.so"))
    for _ in range(3):
        with pytest.raises(RuntimeError, match="none.so is missing"):
            append(pk)
        # calls that do not go through it work
        assert pk.version() and pk.block_bytes(pk.CacheDesc(num_blocks=1, num_kv_heads=1, head_size=64)) == 2048
    monkeypatch.setattr(pk, "BINDING_PATH", path)
    with pytest.raises(TypeError, match="CUDA tensor"):
        append(pk)


def test_a_module_that_does_not_load_fails_every_time(pk, monkeypatch, tmp_path):
    bad = tmp_path / "bad.so"
    bad.write_bytes(b"not an object file")
    monkeypatch.setattr(pk, "BINDING_PATH", str(bad))
    for _ in range(3):
        with pytest.raises(ImportError):
            append(pk)


def test_threads_that_come_first_at_once(pk):
    start, errors = threading.Barrier(8), []

    def run():
        start.wait()
        try:
            append(pk)
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=run) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(errors) == 8 and all(isinstance(e, TypeError) and "CUDA tensor" in str(e) for e in errors)


def test_the_module_is_the_running_interpreters(pk, monkeypatch):
    """Its name carries the interpreter's ABI tag, and a build for another interpreter neither takes this one's
    module for its own nor compiles the library again."""
    import importlib.machinery
    import os
    from paged_kv_cache_10_gb300 import build
    assert pk.BINDING_PATH == build.BINDING and os.path.exists(build.BINDING)
    assert pk.BINDING_PATH.endswith("_pkv_binding" + importlib.machinery.EXTENSION_SUFFIXES[0])
    assert importlib.machinery.EXTENSION_SUFFIXES[0] != ".so"
    made = []
    monkeypatch.setattr(build, "BINDING", build.BINDING.replace("_pkv_binding.", "_pkv_binding.other-"))
    monkeypatch.setattr(build, "_compile_binding", lambda: made.append(1))
    monkeypatch.setattr(build, "ThreadPoolExecutor", None)  # compiling the library would need it
    assert build.build() == build.LIB and made == [1]
