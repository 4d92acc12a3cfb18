"""The argument checks of tests/test_serving_abi_cpu.py under the address and
undefined-behaviour sanitizer build of the library's host code."""
from tests.test_sanitizers_cpu import _child, library_san  # noqa: F401


def test_serving_argument_checks_under_sanitizers(library_san):  # noqa: F811
    lib, rt = library_san
    code = ("import sys, pytest\n"
            "import commit_gated_delta_amd as gdn\n"
            "assert gdn.LIB_PATH == %r\n"
            "sys.exit(pytest.main(['-q', '-x', '-p', 'no:cacheprovider', "
            "'tests/test_serving_abi_cpu.py']))\n" % lib)
    r = _child(code, {"LD_PRELOAD": rt, "GDN_LIBRARY": lib})
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
    assert " passed" in r.stdout
