"""Calls of the attention operators at the edge of what the header allows, on the CPU: where
the pieces of a cut item lie in a workspace, whatever 16 bytes it starts on, sizes that pass
64 bits, workspaces sized at the largest call, and the build without torch's headers or beside
another torch."""
import ctypes
import os
import subprocess

import pytest

from rope_attention_gb300 import build, native

PLACES = r"""
#include <cstdio>
#include "attn_join.cuh"
int main() {
  for (int G : {1, 7, 152, 160})
    for (int NR : {16, 64, 256})
      for (int Dv : {16, 48, 128, 512})
        for (uintptr_t base : {0x10000u, 0x10010u}) {
          ra::JoinParams j{};
          j.NR = NR;
          ra::join_place(&j, reinterpret_cast<uint8_t*>(base), G);
          const uintptr_t meta = reinterpret_cast<uintptr_t>(j.meta), stats = reinterpret_cast<uintptr_t>(j.stats),
                          parts = reinterpret_cast<uintptr_t>(j.parts);
          const uintptr_t end = parts + static_cast<uintptr_t>(G) * 2 * NR * Dv * 4;
          const bool apart = base <= meta && meta + G * 32 <= stats && stats + G * 2 * NR * 16 <= parts;
          printf("%d %d %d %d\n", apart, static_cast<int>(stats % 16), static_cast<int>(parts % 32),
                 end <= base + ra::join_bytes(G, NR, Dv));
        }
}
"""


@pytest.fixture(scope="module")
def nvcc():
    try:
        return build.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")


def host_program(nvcc, tmp_path, source):
    """The lines that a host program over the kernels' headers prints."""
    src, exe = os.path.join(tmp_path, "t.cu"), os.path.join(tmp_path, "t")
    with open(src, "w") as f:
        f.write(source)
    r = subprocess.run([nvcc, src, "-o", exe, "-std=c++17", *build.ARCH, "-I", build.INCLUDE, "-I", build.CSRC, "-cudart", "static"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()


def test_pieces_lie_on_32_bytes_in_a_workspace_on_any_16(nvcc, tmp_path):
    lines = host_program(nvcc, tmp_path, PLACES)
    assert len(lines) == 96 and set(lines) == {"1 0 0 1"}


# ---------------------------------------------------------------- sizes whose products pass 64 bits
A16 = 0x10000  # 16-byte aligned placeholder address (never dereferenced)


@pytest.fixture()
def validating():
    build.build()
    lib = native.load()
    lib.ra_test_validate_only(1)
    yield lib
    lib.ra_test_validate_only(0)


def read_params(**kw):
    base = dict(B=2, N=2, S=5, Dkv=192, Dv=128, rope_size=64, variant=2, cache_mode=native.RA_CACHE_PA_BNSD, block_num=8,
                block_size=32, kv_dtype=native.RA_BF16, k_cache_dtype=native.RA_BF16, ckv_cache_dtype=native.RA_BF16, epsilon=1e-5)
    return native.KvRmsNormRopeCacheParams(**{**base, **kw})


@pytest.mark.parametrize("kw", [
    dict(B=1 << 31, S=1 << 31, N=8),             # B * N * S = 2^65
    dict(B=1 << 31, S=1 << 31, N=4), dict(B=1 << 31, S=1 << 10, N=1),
    # a NORM cache of 2^60 rows, whose bytes wrap to nothing: an empty tensor would hold it
    dict(B=1 << 29, S=1, N=1, cache_mode=native.RA_CACHE_NORM, cache_seq_len=1 << 31, rope_size=8, Dkv=8, Dv=8),
    dict(B=1 << 20, S=1, N=1, cache_mode=native.RA_CACHE_NORM, cache_seq_len=(1 << 20) + 1),
])
def test_read_refuses_sizes_beyond_2_to_the_40(validating, kw):
    p = read_params(**kw)
    st = validating.kv_cache_read(ctypes.byref(p), A16, A16, A16, None, None, None, None, A16, A16, None, None)
    assert st == -1 and "too many" in validating.ra_last_error().decode()
    assert validating.kv_cache_read(ctypes.byref(read_params()), A16, A16, A16, None, None, None, None, A16, A16, None, None) == 0


# ---------------------------------------------------------------- workspaces
@pytest.mark.parametrize("variant,N,heads,new", [(2, 8, 64, 1), (2, 2, 8, 1), (2, 8, 64, 40), (2, 1, 128, 3), (1, 1, 128, 1),
                                                 (1, 1, 16, 2)])
def test_a_workspace_of_the_largest_batch_serves_the_smaller_ones(validating, variant, N, heads, new):
    """The same new tokens a sequence: fewer sequences, or shorter ones, need no more."""
    n = ctypes.c_size_t()

    def need(B, longest):
        c = read_params(variant=variant, N=N, block_num=1 << 16, **(dict(Dkv=576, Dv=512) if variant == 1 else {}))
        p = native.PagedAttentionParams(B=B, total_q=B * new, num_heads=heads, causal=1, softmax_scale=0.1, max_seq_len=longest,
                                        block_table_stride=1 << 12)
        assert validating.paged_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(p), ctypes.byref(n)) == 0
        return n.value

    for longest in (0, 1, 64, 333, 500, 4096, 20000, 131072):
        sizes = [need(B, longest) for B in range(1, 200)]
        assert sizes == sorted(sizes) and sizes[-1] <= 64 << 20, longest
    for B in (1, 3, 19, 20, 38, 40, 160, 1000):
        sizes = [need(B, longest) for longest in (0, 1, 64, 200, 333, 450, 600, 1000, 4096, 20000, 131072)]
        assert sizes == sorted(sizes), B


# ---------------------------------------------------------------- the build
def test_the_library_builds_without_the_headers_of_the_binding(monkeypatch, tmp_path, capsys):
    """nvcc alone makes the library: what only the binding needs may be missing."""
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / build.LIB_NAME))
    monkeypatch.setattr(build, "CALLS_PATH", str(tmp_path / "calls.so"))
    monkeypatch.setattr(build.shutil, "which", lambda name: None if name == "g++" else "/bin/" + name)
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")
    ran = []

    def run(cmd, **kw):
        if cmd[0] == "g++":
            raise FileNotFoundError("g++")
        ran.append(cmd[0])
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    assert build.build() == build.LIB_PATH and os.path.exists(build.LIB_PATH) and not os.path.exists(build.CALLS_PATH)
    assert len(ran) == len(build.SOURCES) + 1 and "g++" in capsys.readouterr().err
    assert build.up_to_date()
    build.build()
    assert len(ran) == len(build.SOURCES) + 1


def test_a_binding_built_for_another_torch_is_not_taken():
    """The module's name holds the interpreter and the torch that it was compiled for."""
    import torch

    assert torch.__version__ in os.path.basename(build.CALLS_PATH)


@pytest.mark.parametrize("text,version", [("__version__ = '2.9.1+cu130'\n", "2.9.1+cu130"),
                                          ('x = 1\n__version__: str = "3.0"\n', "3.0"), ("", "unknown"), (None, "unknown")])
def test_a_torch_without_a_plain_version_file_stops_nothing(monkeypatch, tmp_path, text, version):
    if text is not None:
        (tmp_path / "version.py").write_text(text)
    monkeypatch.setattr(build, "_torch_root", lambda: str(tmp_path))
    assert build._torch_version() == version


def test_a_missing_binding_says_what_its_build_lacks(monkeypatch):
    build.build()
    monkeypatch.setattr(native, "_CALLS", None)
    monkeypatch.setattr(native, "CALLS_PATH", "/nowhere/calls.so")
    monkeypatch.setattr(build, "calls_missing", lambda: "no headers here", raising=False)
    with pytest.raises(FileNotFoundError, match="no headers here"):
        native.packed_attention_params(None, None, None, None)
