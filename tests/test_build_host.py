"""The build on the CPU: what the C library needs, and what only the extension module on PyTorch tensors does."""
import os
import re
import subprocess

import pytest

from mixed_bitrate_quantized_amd import build


@pytest.fixture()
def small(monkeypatch, tmp_path):
    """A build of the host sources alone into a folder of its own."""
    monkeypatch.setattr(build, "HIP_SOURCES", ())
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libexq.so"))
    monkeypatch.setattr(build, "TORCH_LIB", str(tmp_path / "_exq_torch.so"))
    return tmp_path


def broken_extension(monkeypatch, where):
    source = where / "broken.cpp"
    source.write_text("#include <no_such_header.h>\n")
    monkeypatch.setattr(build, "TORCH_SOURCE", str(source))
    monkeypatch.setattr(build, "_torch_flags", lambda: ([], []))


def test_the_library_is_linked_where_the_extension_does_not_compile(small, monkeypatch):
    """PyTorch without Python's headers, or with headers that do not compile: the C library is there, the failure is told."""
    broken_extension(monkeypatch, small)
    with pytest.raises(RuntimeError, match="broken.cpp"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.TORCH_LIB)


def test_the_package_loads_the_library_without_the_extension(small, monkeypatch):
    """Loading the package builds what is missing; without the extension module KVCache says so, the rest works."""
    import mixed_bitrate_quantized_amd as exq
    broken_extension(monkeypatch, small)
    monkeypatch.setattr(exq, "LIB_PATH", build.LIB)
    monkeypatch.setattr(exq, "_PKG", str(small))

    class Loaded(Exception):
        pass

    def stop(path):
        assert os.path.exists(path)
        raise Loaded

    monkeypatch.setattr(exq.ctypes, "CDLL", stop)   # (host sources alone: nothing to bind)
    with pytest.raises(Loaded):
        exq._load()
    with pytest.raises(RuntimeError, match="broken.cpp"):
        exq._tensor_calls()


def test_a_library_that_does_not_compile_ends_the_build(small, monkeypatch):
    source = small / "broken_host.cpp"
    source.write_text("#error no\n")
    monkeypatch.setattr(build, "HOST_SOURCES", (str(source),))
    with pytest.raises(RuntimeError, match="broken_host.cpp"):
        build.build()
    assert not os.path.exists(build.LIB)


def test_parts_are_stored_and_waited_for_before_they_are_counted(tmp_path):
    """In every attention kernel as compiled: the stores of a part, the wait for them, the barrier, the one count."""
    listing = str(tmp_path / "cache.s")
    cmd = [build.hipcc()] + build.HIPCC_FLAGS + ["-S", "--cuda-device-only", "-o", listing, os.path.join(build.CSRC, "exq_cache.hip")]
    subprocess.run(cmd, check=True, capture_output=True)
    kernels, name = {}, None
    with open(listing) as f:
        for line in f:
            label = re.match(r"(\w*attend_kernel\w*):", line)
            if label:
                name = label.group(1)
            if line.startswith(".Lfunc_end"):
                name = None
            if name:
                line = line.strip()
                for letter, pattern in (("S", r"global_store\w* .*\bsc1\b"), ("W", r"s_waitcnt.*\bvmcnt\(0\)"), ("B", "s_barrier"),
                                        ("C", "global_atomic_add")):
                    if re.match(pattern, line):
                        kernels[name] = kernels.get(name, "") + letter
    assert len(kernels) >= 20
    for name, order in kernels.items():
        assert order.count("C") == 1 and re.search("S+W+BC", order), (name, order)
