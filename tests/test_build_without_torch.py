"""What needs no PyTorch works without it: building the library, plans' host side and
the page bookkeeping.  Each check runs in a process of its own in which importing torch fails."""
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


def test_page_bookkeeping_and_import_star():
    out, _ = without_torch("""
        from block_causal_attention_b200 import *
        p = PagePool(4)
        a = p.open()
        assert p.grow(a, 0, 300) == [] and p.row(a) == [0, 1, 2]
        from block_causal_attention_b200.streaming import PipelinedWindow
        assert PipelinedWindow(2, 1, 24, 1, 8, 8, 2, 1, 1, host_only=True).ranges(1) == (1, 1)
        try:
            PagedCache(2, 1, 24, 4, host_only=True)
        except ImportError:
            print("done")
        """)
    assert out.endswith("done\n")
