"""What needs no PyTorch works without it: building the library and plans' host side.  Each check
runs in a process of its own in which importing torch fails."""
import os
import subprocess
import sys
import textwrap

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def without_torch(code, **env):
    head = "import sys\nsys.modules['torch'] = None\n"
    r = subprocess.run([sys.executable, "-W", "always", "-c", head + textwrap.dedent(code)], cwd=ROOT, text=True,
                       capture_output=True, env={**os.environ, **env}, timeout=900)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout, r.stderr


def test_the_library_is_built_and_used(tmp_path):
    """build() gives the library and says that the paged cache's module was left out."""
    out, err = without_torch(f"""
        from block_causal_attention_b200 import Plan, _abi, build
        build.BINDING = {str(tmp_path / "_paged_binding.so")!r}
        lib = build.build()
        import os
        assert lib == build.LIB and os.path.exists(lib) and not os.path.exists(build.BINDING)
        p = Plan(2, 1, 24, [[2, 2, 8, 8, 0]], host_only=True)
        assert p.info()["num_q"] == 256
        print("done")
        """)
    assert out.endswith("done\n") and "paged" in err and "PyTorch" in err
